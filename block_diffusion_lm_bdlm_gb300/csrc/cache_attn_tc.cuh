// cache_attn_tc.cuh - the attention kernel over the paged 8-bit cache, on the
// 5th-generation tensor cores.
//
// Mathematics. A row's scores are s_j = scale ks_j (q . k8_j) with e4m3 codes
// k8 and one scale ks per page. q is bf16 (8 significant bits) and e4m3 holds
// 4, so q = 2^e (q_hi + q_lo) with both terms in e4m3 and 2^e the row's power-
// of-two scale: the two products on the 8-bit pipe (twice the 16-bit rate) give
// the exact q . k8 (entries below 2^-10 of the row's largest lose bits worth
// 2^-18 of it), and the keys go from the page to the tensor core as they lie
// there. The weights need more range than e4m3 has (a thousandth of a weight
// times a hundred thousand keys counts), so the values are widened to fp16
// (exact) on their way and the weights are fp16: p'_j = 2^(log2 p_j + log2 vs_j
// - mo), with the value scale vs of the page in the exponent, where it costs
// nothing, and an offset mo per row that keeps the largest p' between 2^7 and
// 2^15 (fp16 ends at 2^16; what falls below 2^-24 is 2^-31 of the largest).
// l = sum 2^(s_j - m) is kept in fp32 with an offset m of its own: the sum of
// each page's p' times 2^(mo - m - log2 vs).
//
// Bound. A tile of 128 keys is 32 KB from memory at d = 128: about 1490 clocks
// at the measured copy rate shared by 152 SMs. Its MMAs take about 1040 clocks
// for up to 128 flat rows, so these calls are bound by memory, and calls with
// 256 and more flat rows by the tensor pipe.
//
// Roles (384 threads, one CTA per SM, each role walks the CTA's share alone):
//   warps 0-3, 4-7  softmax groups 0 and 1; one TMEM lane = one flat row. They
//                   also split Q into its two terms, and write the results
//   warp 8          page table, scales and TMA loads of K and V pages (3 stages)
//   warp 9          issues the MMAs (one thread), owns TMEM
//   warps 10-11     widen V from e4m3 to fp16 (2 stages), zero the rows behind
//                   the last key and take out masked NaN
// A unit of up to 128 flat rows is one MMA tile: the two groups take its key
// tiles in turn, each with its own sums, and join them at the end, so that one
// group's softmax runs under the other's MMAs. A larger unit is two MMA tiles,
// one for each group, over the same keys.
// TMEM (512 columns): S0 | S1 | O0 | O1; p' overwrites S as fp16.
// MMAs of one thread run in issue order, so the next S of a group is issued
// right behind the PV that reads the p' it overwrites.
// Every mbarrier wait is bounded (2 s); on a timeout the roles drain and the
// share's record carries BDLM_ERR_TIMEOUT.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include "cache_attn.cuh"
#include "tc_ptx.cuh"

namespace bdlm {
namespace cattn {

constexpr int kThreads = 384;
constexpr int kRegsSoftmax = 224;
constexpr int kRegsOther = 56;
constexpr int kTmemCols = 512;
constexpr int kStages = 3;
constexpr int kScaleSlots = 8;
constexpr uint64_t kTimeoutNs = 2000000000ull;

// barriers
enum : int {
    B_KFULL = 0, B_KEMPTY = 3, B_VFULL = 6, B_VEMPTY = 9,  // rings of 3
    B_WFULL = 12, B_WEMPTY = 14,                           // ring of 2
    B_S = 16, B_P = 18, B_O = 20, B_Q = 22,
    B_SC = 23,                                             // ring of 8: scales written
    B_COUNT = 31
};

template <int D>
struct Smem {
    static constexpr int kT8 = 128 * D;        // bytes of a 128-row e4m3 tile
    static constexpr int kQ = 0;               // group 0 hi, lo, group 1 hi, lo
    static constexpr int kW = 4 * kT8;         // fp16 values, 2 stages of 2 * kT8
    static constexpr int kK = 8 * kT8;         // 3 stages
    static constexpr int kV = kK + kStages * kT8;
    static constexpr int kMisc = kV + kStages * kT8;
    static constexpr int kScale = kMisc;                          // float [8 slots][16]: ks, log2 vs of 16-key groups
    static constexpr int kNan = kScale + kScaleSlots * 64;        // int [4][D]: first key whose value is NaN, per column
    static constexpr int kBar = kNan + 4 * D * 4;
    static constexpr int kWords = kBar + B_COUNT * 8;             // tmem, abort, error, info
    static constexpr int kStart = kWords + 16;                    // Start
    static constexpr int kBytes = kStart + 64;
};
static_assert(Smem<128>::kBytes <= 232448, "shared memory");

// Where the CTA's share begins, found once by the whole CTA.
struct Start {
    long long W, begin, left;
    int C, s, h, m0, kt, bad;
};
static_assert(sizeof(Start) <= 64, "");

// A run of tiles of one unit.
struct Seg {
    int row0, rows, pos0, len;  // the sequence
    int s, h, m0, last, end;    // unit
    int kt0, kt1, cost;
    bool two;                   // two MMA tiles
    __device__ __forceinline__ int tiles() const { return end ? kt1 - kt0 : 0; }
    __device__ __forceinline__ bool whole() const { return kt0 == 0 && kt1 == cost; }
};

struct Walk {
    SeqRows r;
    Unit u;
    int s, h, m0, kt;
    long long left;
    __device__ __forceinline__ void begin(const CacheAttnArgs& a, const Start& st) {
        s = st.s;
        h = st.h;
        m0 = st.m0;
        kt = st.kt;
        left = st.left;
        if (left > 0) {
            r = seq_rows(a.c, a.cu_rows, a.q_pos, a.total_rows, s);
            u = unit_of(a, r, m0);
        }
    }
    __device__ __forceinline__ bool next(const CacheAttnArgs& a, Seg* g) {
        if (left <= 0) return false;
        const int n = left < u.cost - kt ? (int)left : u.cost - kt;
        *g = Seg{r.row0, r.rows, r.pos0, r.len, s, h, m0, u.last, u.end, kt, kt + n, u.cost, u.last - m0 > 128};
        left -= n;
        kt += n;
        if (left > 0) {  // the unit is done
            kt = 0;
            m0 += kUnitRows;
            if (m0 >= r.rows * a.G) {
                m0 = 0;
                if (++h == a.c.Hk) {
                    h = 0;
                    do r = seq_rows(a.c, a.cu_rows, a.q_pos, a.total_rows, ++s);
                    while (r.rows == 0);
                }
            }
            u = unit_of(a, r, m0);
        }
        return true;
    }
};

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t widen2(uint32_t c2) {  // two e4m3 codes -> two fp16
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c2 & 0xffffu), __NV_E4M3);
    return (uint32_t)h.x | (uint32_t)h.y << 16;
}
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// D[tmem] (+)= A[smem] B[smem], e4m3 operands
__device__ __forceinline__ void mma_ss_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Instruction descriptor: D fp32, A and B format 0 (e4m3 for kind::f8f6f4, fp16 for kind::f16), A K-major.
__host__ __device__ constexpr uint32_t idesc_fmt0(int M, int N, int b_mn) {
    return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Descriptor of a K-major e4m3 tile whose rows are D bytes: one 128-byte (D = 128) or 64-byte (D = 64) swizzle row
// each, eight rows a group.
template <int D>
__device__ __forceinline__ uint64_t sdesc_k8(uint32_t saddr) {
    uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)1 << 16;
    d |= (uint64_t)(8 * D >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)(D == 128 ? 2 : 4) << 61;
    return d;
}
// Byte offset of 16-byte chunk c of row r in such a tile.
template <int D>
__device__ __forceinline__ uint32_t swz8(int r, int c) {
    return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&r)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void lds16(uint32_t addr, uint32_t (&v)[4]) {
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr));
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

struct Ctx {
    uint8_t* smem;
    uint32_t sbase, tmem;
    int* words;  // tmem, abort, error, info
    __device__ __forceinline__ uint32_t bar(int base, int i) const { return bars + 8 * (base + i); }
    uint32_t bars;
    __device__ __forceinline__ volatile int* abort() const { return words + 1; }
    // bounded wait; false once any role has given up
    __device__ __forceinline__ bool wait(int base, int i, uint32_t parity) const {
        return tc::mbar_wait(bar(base, i), parity, abort(), kTimeoutNs);
    }
};

// ------------------------------------------------------------ share's begin
// Sum over the threads before this one; *total gets the CTA's sum.
__device__ __forceinline__ long long cta_scan(long long x, long long* total, long long* buf) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) buf[warp] = v;
    __syncthreads();
    long long before = 0, t = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const long long y = buf[w];
        if (w < warp) before += y;
        t += y;
    }
    *total = t;
    __syncthreads();
    return before + v - x;
}

__device__ __forceinline__ long long head_cost(const CacheAttnArgs& a, const SeqRows& r) {
    long long c = 0;
    for (int m0 = 0; m0 < r.rows * a.G; m0 += kUnitRows) c += unit_of(a, r, m0).cost;
    return c;
}

__device__ __forceinline__ void find_start(const CacheAttnArgs& a, Start* st, long long* buf) {
    const int tid = threadIdx.x, n = a.c.n_seqs;
    long long W = 0, before = 0, cost = 0, sum;
    int bad = 0x7fffffff;
    for (int s0 = 0; s0 < n; s0 += kThreads) {
        const int s = s0 + tid;
        cost = 0;
        if (s < n) {
            const SeqRows r = seq_rows(a.c, a.cu_rows, a.q_pos, a.total_rows, s);
            if (!r.ok) bad = imin(bad, s);
            else cost = head_cost(a, r) * a.c.Hk;
        }
        before = W + cta_scan(cost, &sum, buf);
        W += sum;
    }
    if (tid == 0) st->bad = 0x7fffffff;
    __syncthreads();
    if (bad != 0x7fffffff) atomicMin(&st->bad, bad);
    __syncthreads();
    bad = st->bad;
    if (bad != 0x7fffffff) W = 0;
    long long C = W / kMinTiles;
    C = C < 1 ? 1 : C > (long long)gridDim.x ? (long long)gridDim.x : C;
    const int c = (int)blockIdx.x;
    const long long begin = c < C ? share_begin(W, (int)C, c) : 0, end = c < C ? share_begin(W, (int)C, c + 1) : 0;
    if (tid == 0) {
        st->W = W;
        st->C = (int)C;
        st->begin = begin;
        st->left = end - begin;
        st->s = st->h = st->m0 = st->kt = 0;
    }
    __syncthreads();
    if (end > begin) {
        long long base = 0;
        for (int s0 = 0; s0 < n; s0 += kThreads) {
            const int s = s0 + tid;
            if (n > kThreads) {  // more than one pass: the costs again
                cost = s < n ? head_cost(a, seq_rows(a.c, a.cu_rows, a.q_pos, a.total_rows, s)) * a.c.Hk : 0;
                before = base + cta_scan(cost, &sum, buf);
                base += sum;
            }
            if (begin >= before && begin < before + cost) {
                const SeqRows r = seq_rows(a.c, a.cu_rows, a.q_pos, a.total_rows, s);
                const long long per = cost / a.c.Hk;
                long long off = begin - before;
                st->s = s;
                st->h = (int)(off / per);
                off %= per;
                int m0 = 0;
                for (int u; off >= (u = unit_of(a, r, m0).cost); m0 += kUnitRows) off -= u;
                st->m0 = m0;
                st->kt = (int)off;
            }
        }
    }
    __syncthreads();
}

// ----------------------------------------------------------------- producer
// The page ids and scales of four tiles at a time: lane l holds those of the
// 16 keys l % 8 of tile l / 8. Ids are read two batches ahead of the loads
// that need them, scales one, so that their latency is hidden.
struct Batch {
    int h, kt, n, end;  // head, first tile, tiles, end of the unit's keys
    int id;             // -1: no key here; -2: malformed
    float ks, vs;
};

struct BatchWalk {
    Walk w;
    Seg g;
    int kt, left;
    __device__ __forceinline__ bool next(const CacheAttnArgs& a, Batch* b) {
        while (left == 0) {
            if (!w.next(a, &g)) return false;
            left = g.tiles();
            kt = g.kt0;
        }
        const int lane = threadIdx.x & 31;
        b->h = g.h;
        b->kt = kt;
        b->n = imin(4, left);
        b->end = g.end;
        const int key = (kt + (lane >> 3)) * kTileKeys + (lane & 7) * 16;
        b->id = -1;
        if ((lane >> 3) < b->n && key < g.end) {
            const int id = __ldg(a.c.table + (long long)g.s * a.c.max_pages + (key >> a.c.page_shift));
            b->id = id >= 0 && id < a.c.n_pages ? id : -2;
        }
        kt += b->n;
        left -= b->n;
        return true;
    }
};

__device__ __forceinline__ void load_scales(const CacheAttnArgs& a, Batch* b) {
    b->ks = 1.f;
    b->vs = 1.f;
    if (b->id >= 0) {
        const long long unit = (long long)b->id * a.c.Hk + b->h;
        b->ks = __ldg(a.c.k_scale + unit);
        b->vs = __ldg(a.c.v_scale + unit);
    }
}

template <int D>
__device__ __forceinline__ void produce(const Ctx& x, const CacheAttnArgs& a, const Start& st, const CUtensorMap* tk,
                                        const CUtensorMap* tv) {
    using L = Smem<D>;
    const int lane = threadIdx.x & 31;
    const int page = a.c.page, per_page = page / 16;
    BatchWalk bw;
    bw.left = 0;
    bw.w.begin(a, st);
    Batch b0, b1, b2;
    bool h0 = bw.next(a, &b0), h1 = h0 && bw.next(a, &b1), h2;
    if (h0) load_scales(a, &b0);
    uint32_t t = 0;
    bool ok = true;
    while (h0 && ok) {
        if (h1) load_scales(a, &b1);
        h2 = h1 && bw.next(a, &b2);
        if (b0.id == -2) {  // the rows of this sequence become NaN through the key scale
            atomicExch(x.words + 2, DEV_CHECK);
            b0.ks = NAN;
        }
        const float lvs = __log2f(b0.vs);
        for (int i = 0; i < b0.n; ++i, ++t) {
            const uint32_t stage = t % kStages, ph = (t / kStages) & 1, slot = t % kScaleSlots;
            ok = x.wait(B_KEMPTY, stage, ph ^ 1) && x.wait(B_VEMPTY, stage, ph ^ 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const bool mine = (lane >> 3) == i;
            const bool load = mine && b0.id >= 0 && (lane & 7) % per_page == 0;
            const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, load)) * page * D;
            if (mine) {
                float* sc = reinterpret_cast<float*>(x.smem + L::kScale) + slot * 16 + (lane & 7);
                sc[0] = b0.ks;
                sc[8] = lvs;
            }
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(x.bar(B_KFULL, stage), bytes);
                tc::mbar_arrive_expect_tx(x.bar(B_VFULL, stage), bytes);
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(x.bar(B_SC, slot));
            if (load) {
                const uint32_t off = stage * L::kT8 + (lane & 7) * 16 * D;
                tc::tma_load_3d(x.sbase + L::kK + off, tk, x.bar(B_KFULL, stage), 0, 0, b0.id * a.c.Hk + b0.h);
                tc::tma_load_3d(x.sbase + L::kV + off, tv, x.bar(B_VFULL, stage), 0, 0, b0.id * a.c.Hk + b0.h);
            }
            __syncwarp();
        }
        b0 = b1;
        b1 = b2;
        h0 = h1;
        h1 = h2;
    }
    if (!ok) {  // a role gave up: wait for the loads in flight before the CTA ends
        int never = 0;
        for (uint32_t i = t > kStages ? t - kStages : 0; i < t; ++i) {
            tc::mbar_wait(x.bar(B_KFULL, i % kStages), (i / kStages) & 1, &never, kTimeoutNs);
            never = 0;
            tc::mbar_wait(x.bar(B_VFULL, i % kStages), (i / kStages) & 1, &never, kTimeoutNs);
            never = 0;
        }
    }
}

// ------------------------------------------------------------ V: e4m3 -> fp16
template <int D>
__device__ __forceinline__ void widen(const Ctx& x, const CacheAttnArgs& a, const Start& st) {
    using L = Smem<D>;
    constexpr int PER = D / 16;             // 16-byte chunks per key
    constexpr int ROWS = 32 / PER;          // keys per warp and step
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - 10;
    const int c = lane % PER, r0 = lane / PER + warp * ROWS;
    Walk w;
    w.begin(a, st);
    Seg g;
    uint32_t t = 0, seg = 0;
    while (w.next(a, &g)) {
        if (g.tiles() == 0) continue;
        int* nan_first = reinterpret_cast<int*>(x.smem + L::kNan) + (seg & 3) * D;
        ++seg;
        // keys that every row of the unit sees; a NaN among the others must not reach a row that does not see it
        const int all = key_end(g.len, a.block, g.pos0 + g.m0 / a.G);
        for (int kt = g.kt0; kt < g.kt1; ++kt, ++t) {
            const uint32_t stage = t % kStages, ws = t & 1;
            bool ok = x.wait(B_VFULL, stage, (t / kStages) & 1) && x.wait(B_WEMPTY, ws, ((t >> 1) & 1) ^ 1);
            if (!__all_sync(0xffffffffu, ok)) return;
            const uint32_t src = x.sbase + L::kV + stage * L::kT8, dst = x.sbase + L::kW + ws * 2 * L::kT8;
            const int valid = imin(kTileKeys, g.end - kt * kTileKeys);
            const bool check = kt * kTileKeys + valid > all;
            for (int i0 = 0; i0 < kTileKeys; i0 += 8 * ROWS) {
                uint32_t v[4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) lds16(src + swz8<D>(i0 + 2 * ROWS * j + r0, c), v[j]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = i0 + 2 * ROWS * j + r0;
                    if (r >= valid) v[j][0] = v[j][1] = v[j][2] = v[j][3] = 0;
                    if (check) {
                        uint32_t any = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) any |= ((v[j][e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                        if (any)
                            for (int e = 0; e < 16; ++e) {
                                const uint32_t sh = 8 * (e & 3);
                                // the element's word by selection, so that v stays in registers
                                const uint32_t word = e < 4 ? v[j][0] : e < 8 ? v[j][1] : e < 12 ? v[j][2] : v[j][3];
                                if (((word >> sh) & 0x7f) == 0x7f) {
                                    atomicMin(nan_first + 16 * c + e, kt * kTileKeys + r);
                                    const uint32_t m = ~(0xffu << sh);
                                    if (e < 4) v[j][0] &= m; else if (e < 8) v[j][1] &= m;
                                    else if (e < 12) v[j][2] &= m; else v[j][3] &= m;
                                }
                            }
                    }
                    uint32_t h[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        h[2 * e] = widen2(v[j][e]);
                        h[2 * e + 1] = widen2(v[j][e] >> 16);
                    }
                    // 16 columns are two 16-byte chunks of the 64-column half they lie in; the lanes of the upper half
                    // store theirs in the other order, so that eight lanes meet eight bank groups
                    const uint32_t base = dst + (c >> 2) * 16384 + r * 128;
                    const uint32_t u = (2 * c) & 7, a0 = base + ((u ^ (r & 7)) << 4), a1 = base + (((u + 1) ^ (r & 7)) << 4);
                    if (c < 4) {
                        sts16(a0, h[0], h[1], h[2], h[3]);
                        sts16(a1, h[4], h[5], h[6], h[7]);
                    } else {
                        sts16(a1, h[4], h[5], h[6], h[7]);
                        sts16(a0, h[0], h[1], h[2], h[3]);
                    }
                }
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(x.bar(B_VEMPTY, stage));
                tc::mbar_arrive(x.bar(B_WFULL, ws));
            }
        }
    }
}

// ---------------------------------------------------------------------- MMA
template <int D>
__device__ __forceinline__ void issue(const Ctx& x, const CacheAttnArgs& a, const Start& st) {
    using L = Smem<D>;
    constexpr uint32_t id_s = idesc_fmt0(128, kTileKeys, 0), id_o = idesc_fmt0(128, D, 1);
    const uint64_t k8 = sdesc_k8<D>(x.sbase), mn = tc::sdesc_sw128(x.sbase, 16384, 1024);
    Walk w;
    w.begin(a, st);
    Seg g;
    uint32_t t_base = 0, seg = 0, n_p[2] = {0, 0};
    while (w.next(a, &g)) {
        const int nt = g.tiles(), jobs = g.two ? 2 * nt : nt;
        if (nt == 0) continue;
        if (!x.wait(B_Q, 0, seg & 1)) return;
        ++seg;
        tc::tc_fence_after();
        // S of job j: group j & 1; its tile is j (one MMA tile) or j / 2 (two)
        auto issue_s = [&](int j) -> bool {
            const uint32_t t = t_base + (g.two ? j >> 1 : j), stage = t % kStages;
            const int i = j & 1;
            if (!g.two || i == 0) {
                if (!x.wait(B_KFULL, stage, (t / kStages) & 1)) return false;
                tc::tc_fence_after();
            }
            const uint64_t dk = tc::sdesc_add(k8, L::kK + stage * L::kT8);
            const uint64_t dq = tc::sdesc_add(k8, L::kQ + (g.two ? i * 2 * L::kT8 : 0));
#pragma unroll
            for (int k = 0; k < 2 * D / 32; ++k)  // the high terms, then the low ones
                mma_ss_f8(x.tmem + 128 * i, tc::sdesc_add(dq, k * 32 < D ? k * 32 : L::kT8 + k * 32 - D),
                          tc::sdesc_add(dk, k * 32 % D), id_s, k > 0);
            tc::mma_commit(x.bar(B_S, i));
            if (!g.two || i == 1) tc::mma_commit(x.bar(B_KEMPTY, stage));
            return true;
        };
        if (!issue_s(0)) return;
        if (jobs > 1 && !issue_s(1)) return;
        for (int j = 0; j < jobs; ++j) {
            const int i = j & 1;
            const uint32_t t = t_base + (g.two ? j >> 1 : j), ws = t & 1;
            if (!g.two || i == 0) {
                if (!x.wait(B_WFULL, ws, (t >> 1) & 1)) return;
            }
            const uint32_t ph = n_p[i] & 1;
            ++n_p[i];
            if (!x.wait(B_P, i, ph)) return;
            tc::tc_fence_after();
            const uint64_t dv = tc::sdesc_add(mn, L::kW + ws * 2 * L::kT8);
#pragma unroll
            for (int k = 0; k < kTileKeys / 16; ++k)
                tc::mma_ts(x.tmem + 256 + D * i, x.tmem + 128 * i + 8 * k, tc::sdesc_add(dv, 2048 * k), id_o,
                           (j > 1 || k > 0) ? 1u : 0u);
            if (!g.two || i == 1) tc::mma_commit(x.bar(B_WEMPTY, ws));
            if (j + 2 >= jobs) tc::mma_commit(x.bar(B_O, i));  // the group's last; waited for, so it comes last
            if (j + 2 < jobs && !issue_s(j + 2)) return;
        }
        t_base += nt;
    }
}

// ------------------------------------------------------------------ softmax
// Splits flat row m0 + row of the unit into its two e4m3 terms; returns the factor that turns the tensor core's q . k8
// into base-2 scores (NaN for a row that is not finite, so that the row becomes NaN and no other).
template <int D>
__device__ __forceinline__ float split_q(const Ctx& x, const CacheAttnArgs& a, const Seg& g, int m, int row, uint32_t dst,
                                         bool hi, bool lo) {
    using L = Smem<D>;
    const __nv_bfloat16* q = a.q + ((long long)(g.row0 + m / a.G) * a.H + g.h * a.G + m % a.G) * D;
    uint4 v[D / 8];
    const bool live = m < g.last;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) v[i] = live ? __ldg(reinterpret_cast<const uint4*>(q) + i) : make_uint4(0, 0, 0, 0);
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t p = (u[e] << 16) & 0x7fffffffu, r = u[e] & 0x7fff0000u;
            big = p > big ? p : big;
            big = r > big ? r : big;
        }
    }
    const float amax = __uint_as_float(big);
    const float s = is_finite(amax) ? pow2_scale(amax) : 1.f, inv = 1.f / s;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
        uint32_t wh[4], wl[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t ph[2], pl[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint4 y = v[2 * c + (e >> 1)];
                const uint32_t u = (e & 1) ? (k ? y.w : y.z) : (k ? y.y : y.x);
                const float f0 = __uint_as_float(u << 16) * inv, f1 = __uint_as_float(u & 0xffff0000u) * inv;
                ph[k] = narrow2(f0, f1);
                const uint32_t back = widen2(ph[k]);
                const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&back));
                pl[k] = narrow2(f0 - b.x, f1 - b.y);
            }
            wh[e] = ph[0] | ph[1] << 16;
            wl[e] = pl[0] | pl[1] << 16;
        }
        if (hi) sts16(dst + swz8<D>(row, c), wh[0], wh[1], wh[2], wh[3]);
        if (lo) sts16(dst + L::kT8 + swz8<D>(row, c), wl[0], wl[1], wl[2], wl[3]);
    }
    return is_finite(amax) ? a.scale_log2 * s : NAN;
}

// One key tile of one row: scores out of TMEM, p' back into it.
template <int D, int NG>
__device__ __forceinline__ void softmax_tile(const Ctx& x, int i, uint32_t slot, uint32_t tS, uint32_t tO, float cs,
                                             int visible, bool full, bool first, float& m, float& mo, float& l) {
    constexpr int GK = kTileKeys / NG;  // keys per page in a tile
    if (!full) {
        // masked entries become -inf in TMEM first, so that other tiles run no mask code
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t v[32];
            tc::tmem_ld32(tS + 32 * q, v);
            tc::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (32 * q + e >= visible) v[e] = 0xff800000u;
            tc::tmem_st32(tS + 32 * q, v);
        }
        tc::tmem_st_wait();
    }
    uint32_t r[4][32];
#pragma unroll
    for (int q = 0; q < 4; ++q) tc::tmem_ld32(tS + 32 * q, r[q]);
    const float* sc = reinterpret_cast<const float*>(x.smem + Smem<D>::kScale) + slot * 16;
    float ks[NG], lv[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        ks[g] = cs * sc[g * (8 / NG)];
        lv[g] = sc[8 + g * (8 / NG)];
    }
    tc::tmem_ld_wait();
    float mx = -INFINITY, mxo = -INFINITY;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        float c0 = -INFINITY, c1 = -INFINITY;
#pragma unroll
        for (int e = 0; e < GK; e += 4) {
            const int k = g * GK + e;
            c0 = tc::fmax3(c0, __uint_as_float(r[k >> 5][k & 31]), __uint_as_float(r[(k + 1) >> 5][(k + 1) & 31]));
            c1 = tc::fmax3(c1, __uint_as_float(r[(k + 2) >> 5][(k + 2) & 31]), __uint_as_float(r[(k + 3) >> 5][(k + 3) & 31]));
        }
        const float y = fmaxf(c0, c1) * ks[g];
        mx = fmaxf(mx, y);
        mxo = fmaxf(mxo, y + lv[g]);
    }
    if (mx > m + 8.f) {
        l *= ex2f(m - mx);
        m = mx;
    }
    const bool move = mxo > mo + 15.f;
    float alpha = 1.f;
    if (move) {
        alpha = ex2f(mo - (mxo - 7.f));
        mo = mxo - 7.f;
    }
    if (!first && __any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tc::tmem_ld32(tO + 32 * q, o);
            tc::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tc::tmem_st32(tO + 32 * q, o);
        }
    }
    const float m_use = m == -INFINITY ? 0.f : m, mo_use = mo == -INFINITY ? 0.f : mo;
    uint32_t pk[2][32];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const float b = lv[g] - mo_use;
        const float2 a2 = make_float2(ks[g], ks[g]), b2 = make_float2(b, b);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < GK; e += 2) {
            const int k = g * GK + e;
            const float2 y = tc::fma2(make_float2(__uint_as_float(r[k >> 5][k & 31]), __uint_as_float(r[k >> 5][(k & 31) + 1])), a2, b2);
            const float2 p = make_float2(ex2f(y.x), ex2f(y.y));
            sum = tc::add2(sum, p);
            pk[k >> 6][(k & 63) >> 1] = pack_h2(p.x, p.y);
        }
        // the page's share of l; where its value scale is so small that p' may have fallen below what fp32 holds, l
        // takes the weights themselves
        const float shift = b + m_use;
        if (__any_sync(0xffffffffu, shift < -60.f)) {
            sum = make_float2(0.f, 0.f);
            for (int e = 0; e < GK; e += 2) {
                const int k = g * GK + e;
                float v0, v1;
                uint32_t s0, s1;
                // the scores again, out of the registers' copy in TMEM (p' is stored below)
                asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=r"(s0), "=r"(s1) : "r"(tS + k));
                tc::tmem_ld_wait();
                v0 = __uint_as_float(s0);
                v1 = __uint_as_float(s1);
                sum.x += ex2f(fmaf(v0, ks[g], -m_use));
                sum.y += ex2f(fmaf(v1, ks[g], -m_use));
            }
            l += sum.x + sum.y;
        } else {
            l = fmaf(sum.x + sum.y, ex2f(-shift), l);
        }
    }
    tc::tmem_st32(tS, pk[0]);
    tc::tmem_st32(tS + 32, pk[1]);
    tc::tmem_st_wait();
    tc::tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(x.bar(B_P, i));
}

// Writes 32 columns of a row: normalised values v.
template <int D>
__device__ __forceinline__ void store_cols(const CacheAttnArgs& a, const Seg& g, int m, int q, const float (&v)[32],
                                           float* slot, int slot_r) {
    if (slot) {
        float4* dst = reinterpret_cast<float4*>(slot) + (long long)(8 * q) * slot_r + (m - g.m0);
#pragma unroll
        for (int e = 0; e < 8; ++e) dst[(long long)e * slot_r] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        return;
    }
    const long long at = ((long long)(g.row0 + m / a.G) * a.H + g.h * a.G + m % a.G) * D + 32 * q;
    if (a.o_f32) {
        float4* dst = reinterpret_cast<float4*>(a.o_f32 + at);
#pragma unroll
        for (int e = 0; e < 8; ++e) dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
    } else {
        uint4* dst = reinterpret_cast<uint4*>(a.o + at);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            dst[e] = make_uint4(pack_bf2(v[8 * e], v[8 * e + 1]), pack_bf2(v[8 * e + 2], v[8 * e + 3]),
                                pack_bf2(v[8 * e + 4], v[8 * e + 5]), pack_bf2(v[8 * e + 6], v[8 * e + 7]));
    }
}

template <int D, int NG>
__device__ __forceinline__ void softmax(const Ctx& x, const CacheAttnArgs& a, const Start& st) {
    using L = Smem<D>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = x.tmem + 128 * i + lane_base, tO = x.tmem + 256 + D * i + lane_base;
    const int slot_r = slot_rows(a.total_rows, a.G);
    Walk w;
    w.begin(a, st);
    Seg g;
    uint32_t t_base = 0, seg = 0, n_s = 0, n_o = 0;
    bool ok = true;  // warp-uniform; the loops run on without waiting once it is false
    while (w.next(a, &g)) {
        const int nt = g.tiles();
        const int m = g.m0 + (g.two ? 128 * i : 0) + row;  // this thread's flat row
        const bool live = m < g.last;
        float* slot = g.whole() ? nullptr : slot_at(a.scratch, 2 * (int)blockIdx.x + (g.kt0 > 0 ? 0 : 1), slot_r, D);
        if (nt == 0) {  // rows without keys
            if (live && (g.two || i == 0)) {
                const float v[32] = {};
                for (int q = 0; q < D / 32; ++q) store_cols<D>(a, g, m, q, v, nullptr, 0);
                a.lse[(long long)(g.h * a.G + m % a.G) * a.total_rows + g.row0 + m / a.G] = -INFINITY;
            }
            continue;
        }
        // Q of the unit: with one MMA tile group 0 writes the high terms, group 1 the low ones
        const float cs = split_q<D>(x, a, g, m, row, x.sbase + L::kQ + (g.two ? i * 2 * L::kT8 : 0), g.two || i == 0, g.two || i == 1);
        tc::fence_proxy_async_smem();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(x.bar(B_Q, 0));

        const int end = live ? key_end(g.len, a.block, g.pos0 + m / a.G) : 0;
        const int full_end = __shfl_sync(0xffffffffu, end, 0);  // the warp's first row sees the fewest keys
        const bool warp_live = __shfl_sync(0xffffffffu, (int)live, 0);
        const int step = g.two ? 1 : 2, first = g.two ? 0 : i;
        float mm = -INFINITY, mo = -INFINITY, l = 0.f;
        for (int j = first; j < nt; j += step) {
            const uint32_t t = t_base + j, slot_no = t % kScaleSlots;
            if (ok) ok = __all_sync(0xffffffffu, x.wait(B_S, i, n_s & 1) && x.wait(B_SC, slot_no, (t / kScaleSlots) & 1));
            ++n_s;
            tc::tc_fence_after();
            const int k0 = (g.kt0 + j) * kTileKeys;
            if (warp_live && ok) {
                softmax_tile<D, NG>(x, i, slot_no, tS, tO, cs, end - k0, k0 + kTileKeys <= full_end, j == first, mm, mo, l);
            } else if (lane == 0) {
                tc::mbar_arrive(x.bar(B_P, i));
            }
        }
        const bool mine = nt > first;  // the group had a tile
        if (mine) {
            if (ok) ok = __all_sync(0xffffffffu, x.wait(B_O, i, n_o & 1));
            ++n_o;
        }
        tc::tc_fence_after();
        int* nan_first = reinterpret_cast<int*>(x.smem + L::kNan) + (seg & 3) * D;
        ++seg;
        t_base += nt;
        if (g.two) {
            // o = O 2^(mo - m) / l
            const bool some = l != 0.f;  // NaN counts as something
            const float f = some ? ex2f(mo - mm) / l : 0.f;
            const float l2 = some ? mm + __log2f(l) : -INFINITY;
            for (int q = 0; q < D / 32; ++q) {
                uint32_t o[32];
                tc::tmem_ld32(tO + 32 * q, o);
                tc::tmem_ld_wait();
                float v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    v[e] = some ? __uint_as_float(o[e]) * f : 0.f;
                    if (nan_first[32 * q + e] < end) v[e] = NAN;
                }
                if (live) store_cols<D>(a, g, m, q, v, slot, slot_r);
            }
            if (live) {
                if (slot) slot[(long long)slot_r * D + m - g.m0] = l2;
                else a.lse[(long long)(g.h * a.G + m % a.G) * a.total_rows + g.row0 + m / a.G] = l2 * 0.69314718055994531f;
            }
            tc::tc_fence_before();
        } else {
            // the groups exchange their sums through their S columns (same lanes) and each writes half of the columns
            tmem_st4(tS, __float_as_uint(mm), __float_as_uint(mo), __float_as_uint(l), 0u);
            tc::tmem_st_wait();
            tc::tc_fence_before();
            softmax_sync();
            tc::tc_fence_after();
            uint32_t ot[4];
            tmem_ld4(x.tmem + 128 * (i ^ 1) + lane_base, ot);
            tc::tmem_ld_wait();
            const float m1 = __uint_as_float(ot[0]), mo1 = __uint_as_float(ot[1]), l1 = __uint_as_float(ot[2]);
            const float mj = fmaxf(mm, m1), moj = fmaxf(mo, mo1);
            const float lj = (mm == -INFINITY && l == 0.f ? 0.f : l * ex2f(mm - mj)) + (m1 == -INFINITY && l1 == 0.f ? 0.f : l1 * ex2f(m1 - mj));
            const bool some = lj != 0.f;
            const float f = some ? ex2f(moj - mj) / lj : 0.f;
            // this group's and the other's factor; a group without a tile or a row without keys in it adds nothing
            const bool use0 = l != 0.f && mine, use1 = l1 != 0.f && nt > (first ^ 1);
            const float f0 = use0 ? f * ex2f(mo - moj) : 0.f, f1 = use1 ? f * ex2f(mo1 - moj) : 0.f;
            const float l2 = some ? mj + __log2f(lj) : -INFINITY;
            const uint32_t tO1 = x.tmem + 256 + D * (i ^ 1) + lane_base;
            for (int q = i * (D / 64); q < (i + 1) * (D / 64); ++q) {
                uint32_t o[32], o1[32];
                tc::tmem_ld32(tO + 32 * q, o);
                tc::tmem_ld32(tO1 + 32 * q, o1);
                tc::tmem_ld_wait();
                float v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    v[e] = (use0 ? __uint_as_float(o[e]) * f0 : 0.f) + (use1 ? __uint_as_float(o1[e]) * f1 : 0.f);
                    if (nan_first[32 * q + e] < end) v[e] = NAN;
                }
                if (live) store_cols<D>(a, g, m, q, v, slot, slot_r);
            }
            if (live && i == 0) {
                if (slot) slot[(long long)slot_r * D + m - g.m0] = l2;
                else a.lse[(long long)(g.h * a.G + m % a.G) * a.total_rows + g.row0 + m / a.G] = l2 * 0.69314718055994531f;
            }
            tc::tc_fence_before();
        }
        // The next unit's Q may be written once both groups are done with this one. The widening warps are at most two
        // tiles ahead of the PV products, so they come back to these words only after three more units have begun.
        softmax_sync();
        if (threadIdx.x < D) nan_first[threadIdx.x] = 0x7fffffff;
    }
}

// ------------------------------------------------------------------- kernel
template <int D, int NG>
__global__ void __launch_bounds__(kThreads, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const CacheAttnArgs a) {
    using L = Smem<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Ctx x;
    x.smem = smem;
    x.sbase = tc::smem_addr(smem);
    x.bars = x.sbase + L::kBar;
    x.words = reinterpret_cast<int*>(smem + L::kWords);
    Start* st = reinterpret_cast<Start*>(smem + L::kStart);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = tid; i < 4 * D; i += kThreads) reinterpret_cast<int*>(smem + L::kNan)[i] = 0x7fffffff;
    if (tid == 0) {
        x.words[1] = x.words[2] = x.words[3] = 0;
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(x.bar(B_KFULL, s), 1);
            tc::mbar_init(x.bar(B_KEMPTY, s), 1);
            tc::mbar_init(x.bar(B_VFULL, s), 1);
            tc::mbar_init(x.bar(B_VEMPTY, s), 2);  // lane 0 of both widening warps
        }
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(x.bar(B_WFULL, s), 2);
            tc::mbar_init(x.bar(B_WEMPTY, s), 1);
            tc::mbar_init(x.bar(B_S, s), 1);
            tc::mbar_init(x.bar(B_P, s), 4);  // lane 0 of each warp of the group
            tc::mbar_init(x.bar(B_O, s), 1);
        }
        tc::mbar_init(x.bar(B_Q, 0), 8);
        for (int s = 0; s < kScaleSlots; ++s) tc::mbar_init(x.bar(B_SC, s), 1);
        tc::fence_barrier_init();
    }
    if (warp == 9) {
        tc::tmem_alloc(tc::smem_addr(x.words), kTmemCols);
        tc::tmem_relinquish();
    }
    if (warp == 8 && lane == 0) {
        tc::prefetch_tmap(&tk);
        tc::prefetch_tmap(&tv);
    }
    find_start(a, st, reinterpret_cast<long long*>(smem));  // the scan's 96 bytes lie where Q will
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    x.tmem = (uint32_t)x.words[0];
    const bool aligned = (x.sbase & 1023u) == 0;  // the swizzled tiles need it; a launch that has not is refused
    if (tid == 0 && !aligned) x.words[1] = 1;
    if (st->left > 0 && aligned) {
        if (warp >= 8) {
            tc::regs_dec<kRegsOther>();
            if (warp == 8) produce<D>(x, a, *st, &tk, &tv);
            else if (warp == 9) {
                if (lane == 0) issue<D>(x, a, *st);
                __syncwarp();
            } else widen<D>(x, a, *st);
        } else {
            tc::regs_inc<kRegsSoftmax>();
            softmax<D, NG>(x, a, *st);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc::tc_fence_after();
        tc::tmem_dealloc(x.tmem, kTmemCols);
    }
    if (tid == 0) {
        ShareRec r{};
        r.W = st->W;
        r.C = st->C;
        if (st->left > 0) {
            const SeqRows q = seq_rows(a.c, a.cu_rows, a.q_pos, a.total_rows, st->s);
            r.row0 = q.row0;
            r.rows = q.rows;
            r.pos0 = q.pos0;
            r.len = q.len;
            r.head = st->h;
            r.m0 = st->m0;
            r.kt0 = st->kt;
            r.cost = unit_of(a, q, st->m0).cost;
        }
        r.error = x.words[1] ? DEV_TIMEOUT : st->bad != 0x7fffffff ? DEV_CHECK : x.words[2];
        r.info = st->bad != 0x7fffffff ? st->bad : (int)blockIdx.x;
        share_recs(a.scratch)[blockIdx.x] = r;
    }
}

// ---------------------------------------------------------------- host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// The pages of all heads as (D, page, n_pages * Hk) bytes; a box is one page of one head.
template <int D>
bool make_map(CUtensorMap* m, const CacheView& c, const void* base) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)c.page, (cuuint64_t)c.n_pages * c.Hk};
    const cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)D * c.page};
    const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)c.page, 1};
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NG>
cudaError_t launch_ng(const CacheAttnArgs& a, int ctas, cudaStream_t st) {
    CUtensorMap tk, tv;
    if (!make_map<D>(&tk, a.c, a.c.k) || !make_map<D>(&tv, a.c, a.c.v)) return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<D, NG>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
    if (e != cudaSuccess) return e;
    cache_attn_kernel<D, NG><<<ctas, kThreads, Smem<D>::kBytes, st>>>(tk, tv, a);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const CacheAttnArgs& a, int ctas, cudaStream_t st) {
    switch (a.c.page) {
        case 16: return launch_ng<D, 8>(a, ctas, st);
        case 32: return launch_ng<D, 4>(a, ctas, st);
        case 64: return launch_ng<D, 2>(a, ctas, st);
        default: return launch_ng<D, 1>(a, ctas, st);
    }
}

}  // namespace cattn
}  // namespace bdlm
