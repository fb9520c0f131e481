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
// nothing, and an offset mo per row that keeps the largest p' between 2^3 and
// 2^15 (fp16 ends at 2^16; what falls below 2^-24 is 2^-27 of the largest).
// l = sum 2^(s_j - m) is kept in fp32 with an offset m of its own: the sum of
// each page's p' times 2^(mo - m - log2 vs).
//
// Bound. A tile of 128 keys is 32 KB from memory at d = 128: about 1430 clocks
// at the measured copy rate shared by 152 SMs. Its MMAs take 1024 clocks for up
// to 128 flat rows, so these calls are bound by memory, and calls with 256 and
// more flat rows by the tensor pipe.
//
// Measured (32 query heads, 8 kv heads, d = 128, whole calls with the merge):
// 64 single rows over 512 to 30912 keys 210 us (4.5 TB/s; a copy of the bytes
// 139), 64 blocks of 32 rows over the same 233 us (1035 TFLOP/s), 64 rows over
// 131072 keys 139 us (990 TFLOP/s), 3 prompts of 5000 to 9000 rows 956 us (890
// TFLOP/s). A tile of a one-tile unit takes 1500 clocks, of a two-tile unit
// 2900 for both: softmax 1450, PV and the next S 1024, four hand-overs 400, one
// after the other, since TMEM has no room for a third S nor shared memory for
// p'. Halving S (64 keys at a time) would break that chain, but 8-bit MMAs with
// N = 64 take 384 clocks instead of 256 for the same work (they read more from
// shared memory than they multiply). Tiles whose offsets move cost 1600 clocks
// more; a unit's query split 2500 to 8000, its results 3500 to 8000, most of it
// the fetching of code that runs once. O is rescaled 64 columns at a time, after p'
// has left its registers (956 against 969 us for the prompts). Tried: sixteen softmax warps, two to a
// row, with shared offsets: 269 and 354 us for the first two calls above when
// eight warps of 64 keys took 216 and 251.
//
// Roles (512 threads, one CTA per SM, each role walks the CTA's share alone):
//   warps 0-3, 4-7  softmax groups 0 and 1; one TMEM lane = one flat row. They
//                   also split Q into its two terms, and write the results
//   warp 8          page table, scales and TMA loads of K (3 stages) and V (2)
//   warp 9          issues the MMAs (one elected lane), owns TMEM
//   warps 10-11     spare
//   warps 12-15     widen V from e4m3 to fp16 (2 stages), zero the rows behind
//                   the last key and take out masked NaN
// A unit of up to 128 flat rows is one MMA tile: group i takes keys 64 i .. of
// every key tile, with sums of its own and O_i, which are joined at the end.
// Two S buffers take turns, so that a tile's softmax runs under the MMAs of
// its neighbours, and the next tile's scores come out of TMEM under this one's
// last steps. A larger unit is two MMA tiles over the same keys, one for each
// group.
// TMEM (512 columns): S0 | S1 | O0 | O1; p' overwrites S as fp16.
// MMAs of one thread run in issue order, so the next S of a buffer is issued
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

constexpr int kThreads = 512;
constexpr int kSoftmax = 256;
// 16 warps at 128 registers each, redistributed. What a role keeps beyond its registers would be spilled to an L1 that
// shared memory leaves next to no room.
constexpr int kRegsSoftmax = 176;
constexpr int kRegsOther = 80;
static_assert(8 * kRegsSoftmax + 8 * kRegsOther <= 16 * 128, "registers");
constexpr int kTmemCols = 512;
constexpr int kStages = 3;  // of K; V has two as e4m3 and two as fp16
constexpr int kScaleSlots = 6;
constexpr uint64_t kTimeoutNs = 2000000000ull;

// Barriers. Tiles are numbered through the CTA's share; t is a tile's number.
enum : int {
    B_KFULL = 0,                // t % 3
    B_VFULL = 3, B_VEMPTY = 5,  // t & 1
    B_S0 = 7,                   // t % 3: the first S of a unit of two MMA tiles
    B_S1 = 10,                  // t % 3: the tile's last S; it also frees the K stage
    B_P = 13,                   // 2 (t & 1) + i: p' of group i in TMEM; for group 0 also V in fp16
    B_PV = 17,                  // t & 1: the tile's products with V; frees the fp16 stage
    B_Q = 19,
    B_COUNT = 20
};

template <int D>
struct Smem {
    static constexpr int kT8 = 128 * D;        // bytes of a 128-row e4m3 tile
    static constexpr int kQ = 0;               // group 0 hi, lo, group 1 hi, lo
    static constexpr int kW = 4 * kT8;         // fp16 values, 2 stages of 2 * kT8
    static constexpr int kK = 8 * kT8;
    static constexpr int kV = kK + kStages * kT8;  // 2 stages
    static constexpr int kMisc = kV + 2 * kT8;
    static constexpr int kScale = kMisc;                          // float [slots][16]: ks, log2 vs of 16-key groups
    static constexpr int kNan = kScale + kScaleSlots * 64;        // int [4][D]: first key whose value is NaN, per column
    static constexpr int kNanAny = kNan + 4 * D * 4;              // int [4]: first key with a NaN in any column
    static constexpr int kBar = kNanAny + 16;
    static constexpr int kWords = kBar + B_COUNT * 8;             // tmem, abort, error, info
    static constexpr int kStart = kWords + 16;                    // Start
    static constexpr int kQExp = kStart + 64;                     // uint8 [256]: exponent of the rows' scale
    static constexpr int kPlace = kQExp + kUnitRows;              // Place of each warp
    static constexpr int kBytes = kPlace + (kThreads / 32) * 128;
};
static_assert(Smem<128>::kBytes <= 232448, "shared memory");

// Where the CTA's share begins, found once by the whole CTA.
struct Start {
    long long per, left;
    int more, C, s, h, m0, off, bad;
};
static_assert(sizeof(Start) <= 64, "");

// A run of tiles of one unit.
struct Seg {
    int row0, pos0, len;  // the sequence
    int s, h, m0, last, end;
    int kt0, kt1;
    bool two, whole;
    __device__ __forceinline__ int tiles() const { return end ? kt1 - kt0 : 0; }
};

struct Place {
    SeqRows r;
    Unit u;
    int s, h, m0, off;
    long long left;
    Seg g;  // the present run
};
static_assert(sizeof(Place) <= 128, "");

// Both are called by whole warps; the warp's lanes write the same values.
__device__ __forceinline__ void begin_share(const CacheAttnArgs& a, const Start& st, Place* p) {
    p->s = st.s;
    p->h = st.h;
    p->m0 = st.m0;
    p->off = st.off;
    p->left = st.left;
    if (st.left > 0) {
        p->r = seq_rows(a.c, a.cu_rows, a.q_pos, a.total_rows, st.s);
        p->u = unit_of(a, p->r, st.m0);
    }
    __syncwarp();
}
// The next run of tiles, into p->g; false behind the last.
__device__ __forceinline__ bool next_run(const CacheAttnArgs& a, Place* p) {
    __syncwarp();
    long long left = p->left;
    bool found = false;
    while (left > 0 && !found) {
        const Unit u = p->u;
        const int off = p->off, c = u.cost(), n = left < c - off ? (int)left : c - off;
        const int kt0 = tile_at(off, u.two, u.lead), kt1 = tile_at(off + n, u.two, u.lead);
        int s = p->s, h = p->h, m0 = p->m0;
        SeqRows r = p->r;
        found = kt1 > kt0;
        __syncwarp();
        if (found) p->g = Seg{r.row0, r.pos0, r.len, s, h, m0, u.last, u.end, kt0, kt1, u.two != 0, kt0 == 0 && kt1 == u.tiles};
        left -= n;
        if (left > 0) {  // the unit is done
            m0 += kUnitRows;
            if (m0 >= r.rows * a.G) {
                m0 = 0;
                if (++h == a.c.Hk) {
                    h = 0;
                    do r = seq_rows(a.c, a.cu_rows, a.q_pos, a.total_rows, ++s);
                    while (r.rows == 0);
                    p->r = r;
                    p->s = s;
                }
                p->h = h;
            }
            p->m0 = m0;
            p->off = 0;
            p->u = unit_of(a, r, m0);
        }
        p->left = left;
        __syncwarp();
    }
    return found;
}

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
// four e4m3 codes -> four fp16
__device__ __forceinline__ void widen4(uint32_t c, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(c));
}
// four fp16 -> four e4m3 codes (nearest even, saturating)
__device__ __forceinline__ uint32_t narrow4(uint32_t lo, uint32_t hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e4m3x2.f16x2 a, %1;\n\tcvt.rn.satfinite.e4m3x2.f16x2 b, %2;\n\t"
        "mov.b32 %0, {a, b};\n\t}"
        : "=r"(r)
        : "r"(lo), "r"(hi));
    return r;
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
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void sts8(uint32_t addr, uint32_t a, uint32_t b) {
    asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void lds8(uint32_t addr, uint32_t& a, uint32_t& b) {
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr));
}
__device__ __forceinline__ void lds16(uint32_t addr, uint32_t (&v)[4]) {
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr));
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ void group_sync(int i) { asm volatile("bar.sync %0, 128;" ::"r"(2 + i) : "memory"); }

template <int N>
struct Const {
    static constexpr int value = N;
};
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
    return p != 0;
}

extern __shared__ __align__(1024) uint8_t g_smem[];
__device__ __forceinline__ uint32_t sbase() { return tc::smem_addr(g_smem); }

template <int D>
struct Ctx {
    using L = Smem<D>;
    uint32_t tmem, base;
    // Values of the role's own: the compiler would else compute what the roles have in common before it branches into
    // them, and carry it through all of them in registers that they do not have.
    __device__ __forceinline__ Ctx own() const {
        Ctx c;
        asm volatile("mov.u32 %0, %1;" : "=r"(c.tmem) : "r"(tmem));
        asm volatile("mov.u32 %0, %1;" : "=r"(c.base) : "r"(base));
        return c;
    }
    __device__ __forceinline__ uint32_t bar(int b, int i) const { return base + L::kBar + 8 * (b + i); }
    static __device__ __forceinline__ int* words() { return reinterpret_cast<int*>(g_smem + L::kWords); }  // tmem, abort, error
    // bounded wait; false once any role has given up
    __device__ __forceinline__ bool wait(int b, int i, uint32_t parity) const {
        return tc::mbar_wait(bar(b, i), parity, words() + 1, kTimeoutNs);
    }
    // The warp's place in the share. It lies in shared memory: every lane of a warp has the same, it changes once per
    // unit, and registers that hold it through the tile loops would be spilled, to an L1 that has next to no room.
    static __device__ __forceinline__ Place* place() { return reinterpret_cast<Place*>(g_smem + L::kPlace + (threadIdx.x >> 5) * 128); }
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

// Cost of one head of sequence s of this lane; the units of long sequences are shared out over the warp.
__device__ __forceinline__ long long head_cost(const CacheAttnArgs& a, const SeqRows& r, bool have) {
    constexpr int kFew = 2;
    const int units = have ? (r.rows * a.G + kUnitRows - 1) / kUnitRows : 0, lane = threadIdx.x & 31;
    long long c = 0;
    if (units <= kFew)
        for (int i = 0; i < units; ++i) c += unit_of(a, r, i * kUnitRows).cost();
    for (unsigned todo = __ballot_sync(0xffffffffu, units > kFew); todo; todo &= todo - 1) {
        const int src = __ffs(todo) - 1, n = __shfl_sync(0xffffffffu, units, src);
        SeqRows q;
        q.rows = __shfl_sync(0xffffffffu, r.rows, src);
        q.len = __shfl_sync(0xffffffffu, r.len, src);
        q.pos0 = __shfl_sync(0xffffffffu, r.pos0, src);
        long long x = 0;
        for (int i = lane; i < n; i += 32) x += unit_of(a, q, i * kUnitRows).cost();
#pragma unroll
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane == src) c = x;
    }
    return c;
}

// The unit of sequence r that holds offset *off of a head's cost, by one whole warp; *off becomes the offset in it.
__device__ __forceinline__ int find_unit(const CacheAttnArgs& a, const SeqRows& r, long long* off) {
    const int lane = threadIdx.x & 31;
    for (int i0 = 0;; i0 += 32) {
        const int m0 = (i0 + lane) * kUnitRows;
        const long long c = m0 < r.rows * a.G ? unit_of(a, r, m0).cost() : 0;
        long long v = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, v > *off);
        if (hit) {
            const int k = __ffs(hit) - 1;
            *off -= __shfl_sync(0xffffffffu, v - c, k);
            return (i0 + k) * kUnitRows;
        }
        const long long all = __shfl_sync(0xffffffffu, v, 31);
        if (all == 0) return 0;  // not reached: the offset lies within the head's cost
        *off -= all;
    }
}

__device__ __forceinline__ void find_start(const CacheAttnArgs& a, Start* st, long long* buf) {
    const int tid = threadIdx.x, n = a.c.n_seqs;
    if (tid == 0) {
        st->left = 0;
        st->bad = 0x7fffffff;
        st->s = st->h = st->m0 = st->off = 0;
    }
    __syncthreads();
    long long W = 0, before = 0, cost = 0, sum;
    SeqRows r{};
    for (int s0 = 0; s0 < n; s0 += kThreads) {
        const int s = s0 + tid;
        bool have = s < n;
        if (have) {
            r = seq_rows(a.c, a.cu_rows, a.q_pos, a.total_rows, s);
            if (!r.ok) atomicMin(&st->bad, s);
            have = r.ok;
        }
        cost = head_cost(a, r, have);
        before = W + cta_scan(cost * a.c.Hk, &sum, buf);
        W += sum;
    }
    // (the scan's barriers order the writes of st->bad)
    const int c = (int)blockIdx.x;
    if (st->bad != 0x7fffffff) W = 0;
    const long long most = W / kMinShare;
    const int C = most < 1 ? 1 : most > (long long)gridDim.x ? (int)gridDim.x : (int)most;
    const long long per = W / C;
    const int more = (int)(W - per * C);
    const long long begin = share_begin(per, more, c), left = c < C ? share_begin(per, more, c + 1) - begin : 0;
    if (tid == 0) {
        st->per = per;
        st->more = more;
        st->C = C;
        st->left = left;
    }
    if (left > 0) {
        long long base = 0;
        for (int s0 = 0; s0 < n; s0 += kThreads) {
            const int s = s0 + tid;
            if (n > kThreads) {  // more than one pass: the costs again
                if (s < n) r = seq_rows(a.c, a.cu_rows, a.q_pos, a.total_rows, s);
                cost = head_cost(a, r, s < n);
                before = base + cta_scan(cost * a.c.Hk, &sum, buf);
                base += sum;
            }
            const bool mine = begin >= before && begin < before + cost * a.c.Hk;
            const unsigned who = __ballot_sync(0xffffffffu, mine);
            if (who) {  // one warp of the CTA
                const int src = __ffs(who) - 1;
                long long off = begin - before;
                int h = 0;
                if (mine)
                    for (; off >= cost; ++h) off -= cost;
                SeqRows q;
                q.rows = __shfl_sync(0xffffffffu, r.rows, src);
                q.len = __shfl_sync(0xffffffffu, r.len, src);
                q.pos0 = __shfl_sync(0xffffffffu, r.pos0, src);
                off = __shfl_sync(0xffffffffu, off, src);
                const int m0 = find_unit(a, q, &off);
                if (mine) {
                    st->s = s;
                    st->h = h;
                    st->m0 = m0;
                    st->off = (int)off;
                }
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
    Place* p;
    int kt, left;
    __device__ __forceinline__ bool next(const CacheAttnArgs& a, Batch* b) {
        while (left == 0) {
            if (!next_run(a, p)) return false;
            left = p->g.tiles();
            kt = p->g.kt0;
        }
        const Seg& g = p->g;
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
__device__ __forceinline__ void produce(const Ctx<D>& x, const CacheAttnArgs& a, const Start& st, const CUtensorMap* tk,
                                        const CUtensorMap* tv) {
    using L = Smem<D>;
    const int lane = threadIdx.x & 31;
    const int page = a.c.page, per_page = page / 16;
    BatchWalk bw;
    bw.left = 0;
    bw.p = x.place();
    begin_share(a, st, bw.p);
    Batch b0, b1, b2;
    bool h0 = bw.next(a, &b0), h1 = h0 && bw.next(a, &b1), h2;
    if (h0) load_scales(a, &b0);
    uint32_t t = 0;
    bool ok = true;
    while (h0 && ok) {
        if (h1) load_scales(a, &b1);
        h2 = h1 && bw.next(a, &b2);
        if (b0.id == -2) {  // the rows of this sequence become NaN through the key scale
            atomicExch(x.words() + 2, DEV_CHECK);
            b0.ks = NAN;
        }
        const float lvs = __log2f(b0.vs);
        for (int i = 0; i < b0.n; ++i, ++t) {
            const uint32_t stage = t % kStages, vs = t & 1, slot = t % kScaleSlots;
            ok = x.wait(B_S1, stage, ((t / kStages) & 1) ^ 1) && x.wait(B_VEMPTY, vs, ((t >> 1) & 1) ^ 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const bool mine = (lane >> 3) == i;
            const bool load = mine && b0.id >= 0 && (lane & 7) % per_page == 0;
            const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, load)) * page * D;
            if (mine) {
                float* sc = reinterpret_cast<float*>(g_smem + L::kScale) + slot * 16 + (lane & 7);
                sc[0] = b0.ks;
                sc[8] = lvs;
            }
            // The scales are written before the arrival on the keys' barrier, which the MMA warp awaits before it issues and
            // commits the S that the softmax warps await: they read them behind it.
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(x.bar(B_KFULL, stage), bytes);
                tc::mbar_arrive_expect_tx(x.bar(B_VFULL, vs), bytes);
            }
            __syncwarp();
            if (load) {
                const uint32_t off = (lane & 7) * 16 * D;
                tc::tma_load_3d(x.base + L::kK + stage * L::kT8 + off, tk, x.bar(B_KFULL, stage), 0, 0, b0.id * a.c.Hk + b0.h);
                tc::tma_load_3d(x.base + L::kV + vs * L::kT8 + off, tv, x.bar(B_VFULL, vs), 0, 0, b0.id * a.c.Hk + b0.h);
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
            if (i + 2 >= t) tc::mbar_wait(x.bar(B_VFULL, i & 1), (i >> 1) & 1, &never, kTimeoutNs);
            never = 0;
        }
    }
}

// ------------------------------------------------------------ V: e4m3 -> fp16
template <int D>
__device__ __forceinline__ void widen(const Ctx<D>& x, const CacheAttnArgs& a, const Start& st) {
    using L = Smem<D>;
    constexpr int PER = D / 16;                  // 16-byte chunks per key
    constexpr int ROWS = 4 * (32 / PER);         // keys that the four warps take at a time
    constexpr int STEPS = kTileKeys / ROWS, HALF = STEPS / 2;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - 12;
    const int c = lane % PER, r0 = lane / PER + warp * (32 / PER);
    // 16 columns are two 16-byte chunks of the 64-column half they lie in; the lanes of the upper half read and store
    // theirs in the other order, so that eight lanes meet eight bank groups. The rows of a thread are ROWS (a multiple of 8)
    // apart, so its swizzle is the same in every step.
    const uint32_t row_dst = x.base + L::kW + (c >> 2) * 16384 + r0 * 128;
    const bool swap = c >= 4;
    const uint32_t src0 = x.base + L::kV + swz8<D>(r0, c) + (swap ? 8 : 0), src1 = src0 ^ 8;
    const uint32_t d0 = row_dst + ((((2 * c + (swap ? 1 : 0)) & 7) ^ (r0 & 7)) << 4);
    const uint32_t d1 = row_dst + ((((2 * c + (swap ? 0 : 1)) & 7) ^ (r0 & 7)) << 4);
    Place* place = x.place();
    begin_share(a, st, place);
    uint32_t t = 0, seg = 0;
    while (next_run(a, place)) {
        if (place->g.tiles() == 0) continue;
        // keys that every row of the unit sees; a NaN among the others must not reach a row that does not see it
        const int all = key_end(place->g.len, a.block, place->g.pos0 + place->g.m0 / a.G), end = place->g.end, kt1 = place->g.kt1;
        for (int kt = place->g.kt0; kt < kt1; ++kt, ++t) {
            const uint32_t ws = t & 1;
            bool ok = x.wait(B_VFULL, ws, (t >> 1) & 1);
            const int valid = imin(kTileKeys, end - kt * kTileKeys);
            const bool check = valid < kTileKeys || kt * kTileKeys + valid > all;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t v[HALF][4];
#pragma unroll
                for (int j = 0; j < HALF; ++j) {
                    const uint32_t from = ws * L::kT8 + (half * HALF + j) * ROWS * D;
                    lds8(src0 + from, v[j][0], v[j][1]);
                    lds8(src1 + from, v[j][2], v[j][3]);
                }
                if (half == 0) {
                    ok = ok && x.wait(B_PV, ws, ((t >> 1) & 1) ^ 1);
                    if (!__all_sync(0xffffffffu, ok)) return;
                }
                if (check) {
#pragma unroll
                    for (int j = 0; j < HALF; ++j) {
                        const int r = (half * HALF + j) * ROWS + r0;
                        if (r >= valid) v[j][0] = v[j][1] = v[j][2] = v[j][3] = 0;
                        uint32_t any = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) any |= ((v[j][e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                        if (any) {
                            int* nan_first = reinterpret_cast<int*>(g_smem + L::kNan) + (seg & 3) * D + 16 * c;
                            atomicMin(reinterpret_cast<int*>(g_smem + L::kNanAny) + (seg & 3), kt * kTileKeys + r);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const uint32_t sh = 8 * (e & 3);
                                if (((v[j][e >> 2] >> sh) & 0x7f) == 0x7f) {
                                    atomicMin(nan_first + (e ^ (swap ? 8 : 0)), kt * kTileKeys + r);
                                    v[j][e >> 2] &= ~(0xffu << sh);
                                }
                            }
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < HALF; ++j) {
                    const uint32_t to = ws * 2 * L::kT8 + (half * HALF + j) * ROWS * 128;
                    uint32_t h[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) widen4(v[j][e], h[2 * e], h[2 * e + 1]);
                    sts16(d0 + to, h[0], h[1], h[2], h[3]);
                    sts16(d1 + to, h[4], h[5], h[6], h[7]);
                }
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(x.bar(B_VEMPTY, ws));
                tc::mbar_arrive(x.bar(B_P, 2 * ws));
            }
        }
        ++seg;
    }
}

// ---------------------------------------------------------------------- MMA
// The whole warp walks the share, and everything that an address or a
// descriptor is made of is warp-uniform to the compiler too (constants, counts
// and results of reductions), so that it keeps them in uniform registers, where
// the MMA reads them; one elected lane issues. The tensor pipe queues little,
// so what stands between two groups of MMAs is kept short: one wait for a
// tile's keys, one for p' of each O (which counts the fp16 values as well) and
// one commit for each S and each PV.
template <int D>
__device__ __forceinline__ void issue(const CacheAttnArgs& a, const Start& st) {
    using L = Smem<D>;
    constexpr uint32_t id_s = idesc_fmt0(128, kTileKeys, 0), id_o = idesc_fmt0(128, D, 1);
    Ctx<D> x;
    x.tmem = 0;  // all of TMEM is this CTA's (the kernel has checked it)
    x.base = sbase();
    const uint64_t k8 = sdesc_k8<D>(sbase()), mn = tc::sdesc_sw128(sbase(), 16384, 1024);
    const bool leader = elect_one();
    auto wait = [&](int base, int i, uint32_t parity) { return __all_sync(0xffffffffu, x.wait(base, i, parity)) != 0; };
    // S of the tile in K stage `stage`, from Q tile qt into S buffer b
    auto issue_s = [&](uint32_t stage, uint32_t qt, uint32_t b, int bar) {
        const uint64_t dk = tc::sdesc_add(k8, L::kK + stage * L::kT8), dq = tc::sdesc_add(k8, L::kQ + qt * 2 * L::kT8);
        if (leader) {
#pragma unroll
            for (int k = 0; k < 2 * D / 32; ++k)  // the high terms, then the low ones
                mma_ss_f8(128 * b, tc::sdesc_add(dq, k * 32 < D ? k * 32 : L::kT8 + k * 32 - D), tc::sdesc_add(dk, k * 32 % D), id_s, k > 0);
            tc::mma_commit(x.bar(bar, stage));
        }
    };
    // N steps of p' (from TMEM column p on) times the fp16 values in stage b from key `key` on, into O buffer o
    auto issue_pv = [&](uint32_t b, uint32_t p, uint32_t o, int key, auto steps, bool fresh) {
        constexpr int N = decltype(steps)::value;
        const uint64_t dv = tc::sdesc_add(mn, L::kW + b * 2 * L::kT8 + key * 128);
        if (leader) {
#pragma unroll
            for (int k = 0; k < N; ++k) tc::mma_ts(256 + D * o, p + 8 * k, tc::sdesc_add(dv, 2048 * k), id_o, (k > 0 || !fresh) ? 1u : 0u);
        }
    };
    auto up = [](uint32_t& stage, uint32_t& ph) {  // the next stage of a ring of three, and its phase
        if (++stage == kStages) {
            stage = 0;
            ph ^= 1;
        }
    };
    Place* place = x.place();
    begin_share(a, st, place);
    uint32_t b = 0, ph = 0;            // t & 1 and (t >> 1) & 1 of the tile whose p' comes next
    uint32_t stage = 0, ks = 0, q = 0;  // the K stage whose keys come next, its phase, and Q's
    while (__any_sync(0xffffffffu, next_run(a, place))) {
        const int nt = __reduce_max_sync(0xffffffffu, place->g.tiles());
        if (nt == 0) continue;
        const int two = __reduce_max_sync(0xffffffffu, (int)place->g.two);
        if (!wait(B_Q, 0, q)) return;
        q ^= 1;
        tc::tc_fence_after();
        if (two) {
            if (!wait(B_KFULL, stage, ks)) return;
            issue_s(stage, 0, 0, B_S0);
            issue_s(stage, 1, 1, B_S1);
            up(stage, ks);
            for (int j = 0; j < nt; ++j) {
                const bool more = j + 1 < nt;
#pragma unroll
                for (uint32_t i = 0; i < 2; ++i) {
                    if (!wait(B_P, 2 * b + i, ph)) return;
                    tc::tc_fence_after();
                    issue_pv(b, 128 * i, i, 0, Const<8>{}, j == 0);
                    if (i == 1 && leader) tc::mma_commit(x.bar(B_PV, b));
                    if (more) {
                        if (i == 0 && !wait(B_KFULL, stage, ks)) return;
                        issue_s(stage, i, i, i == 0 ? B_S0 : B_S1);
                    }
                }
                if (more) up(stage, ks);
                ph ^= b;
                b ^= 1;
            }
        } else {
#pragma unroll 1
            for (int j = 0; j < 2 && j < nt; ++j) {
                if (!wait(B_KFULL, stage, ks)) return;
                issue_s(stage, 0, b ^ j, B_S1);
                up(stage, ks);
            }
            for (int j = 0; j < nt; ++j) {
#pragma unroll
                for (uint32_t i = 0; i < 2; ++i) {  // each half of the keys into its own O
                    if (!wait(B_P, 2 * b + i, ph)) return;
                    tc::tc_fence_after();
                    issue_pv(b, 128 * b + 64 * i, i, 64 * i, Const<4>{}, j == 0);
                }
                if (leader) tc::mma_commit(x.bar(B_PV, b));
                if (j + 2 < nt) {
                    if (!wait(B_KFULL, stage, ks)) return;
                    issue_s(stage, 0, b, B_S1);
                    up(stage, ks);
                }
                ph ^= b;
                b ^= 1;
            }
        }
    }
}

// ------------------------------------------------------------------ softmax
// Splits the unit's rows into their two e4m3 terms and notes the exponents of their power-of-two scales (255 for a row
// that is not finite). Eight values per thread, so that a row is read and reduced by D / 8 lanes; rows behind the last
// one of a warp's 32 are zeros.
template <int D>
__device__ __forceinline__ void split_q(const Ctx<D>& x, const CacheAttnArgs& a, const Seg& g) {
    using L = Smem<D>;
    constexpr int PER = D / 8, ROWS = kSoftmax / PER, BATCH = 4;
    const int chunk = threadIdx.x % PER, r0 = threadIdx.x / PER;
    const int n = g.last - g.m0, padded = (n + 31) & ~31;
    uint8_t* exps = g_smem + L::kQExp;
    const __nv_bfloat16* q = a.q + ((long long)g.row0 * a.H + g.h * a.G) * D + 8 * chunk;
    const int dr = ROWS / a.G, dm = ROWS - dr * a.G;
    int row = (g.m0 + r0) / a.G, rem = g.m0 + r0 - row * a.G, next = r0;
    auto load = [&]() {
        uint4 y = make_uint4(0, 0, 0, 0);
        if (next < n) y = __ldg(reinterpret_cast<const uint4*>(q + ((long long)row * a.H + rem) * D));
        next += ROWS;
        row += dr;
        rem += dm;
        if (rem >= a.G) {
            rem -= a.G;
            ++row;
        }
        return y;
    };
    // four rows at a time, the next four in flight; the loop is not unrolled further, since most of what a first pass
    // through this code costs is fetching the code
    uint4 v[BATCH], w[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) v[i] = load();
#pragma unroll 1
    for (int b = 0; b < padded; b += BATCH * ROWS) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) w[i] = load();
        uint32_t big[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            big[i] = __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu), __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu));
#pragma unroll
        for (int o = PER / 2; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < BATCH; ++i) big[i] = __vmaxu2(big[i], __shfl_xor_sync(0xffffffffu, big[i], o));
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int r = b + i * ROWS + r0;
            const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            const uint32_t top = (uint32_t)imax((int)(big[i] & 0xffffu), (int)(big[i] >> 16)) << 16;
            const bool fine = top < 0x7f800000u;
            const uint32_t sc = fine ? __float_as_uint(pow2_scale(__uint_as_float(top))) : 0x3f800000u;
            // 2^-k for 2^k, -126 <= k <= 120, twice as bf16; the products are exact, and in fp16 too (at most 448, and what
            // fp16 drops is 2^-33 of the row's largest)
            const uint32_t inv2 = __byte_perm(0x7f000000u - sc, 0, 0x3232);
            const __nv_bfloat162 inv = *reinterpret_cast<const __nv_bfloat162*>(&inv2);
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t f[2], h[2], d[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&u[2 * e + k]), inv);
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(&y);
                    f[k] = pack_h2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
                }
                hi[e] = narrow4(f[0], f[1]);
                widen4(hi[e], h[0], h[1]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&f[k]), *reinterpret_cast<const __half2*>(&h[k]));
                    d[k] = *reinterpret_cast<const uint32_t*>(&y);
                }
                lo[e] = narrow4(d[0], d[1]);
            }
            if (r < padded) {
                const uint32_t at = x.base + L::kQ + (r >> 7) * 2 * L::kT8 + swz8<D>(r & 127, chunk >> 1) + 8 * (chunk & 1);
                sts8(at, hi[0], hi[1]);
                sts8(at + L::kT8, lo[0], lo[1]);
                if (chunk == 0) exps[r] = fine ? (uint8_t)(sc >> 23) : (uint8_t)255;
            }
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) v[i] = w[i];
    }
}

// One row's running sums: l = sum 2^(s - m), and O = sum 2^(s + log2 vs - mo) v8.
struct RowSums {
    float m, mo, l;
};

// A factor of scores: not so small that it turns the -inf of a masked key into NaN (NaN stays).
__device__ __forceinline__ float at_least(float x) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(1.17549435e-38f));
    return y;
}

// p' of the 64 keys of a row whose scores were loaded from TMEM column tC on into r; p' goes to the columns from tP on as
// fp16 pairs. NG pages of GK keys each; sc points at the first one's key scale. The row sees the first `visible` keys; `full`: all of the
// warp's rows see all; `first`: the row's O holds nothing yet. `settle(alpha)` waits until O (at tO) may be rescaled, and
// rescales by the power of two alpha what the tile has stored of p' already.
//
// Keys are first taken with the row's present offsets. p' is positive, so a sum of at most 2^15 says that every p' fits
// fp16, and no maximum is needed; it holds for all but a few tiles of a sequence. Where a row of the warp has a larger
// sum or sees its first keys, or a page's value scale is so small that its p' may fall below what fp32 holds, the warp
// takes the keys again: new offsets from their maxima, O and l rescaled, and l from the weights themselves where p' says
// too little. (A sum over 2^15 of 64 keys has a p' of 2^9, which moves mo; the largest is at most 2^4 then, which leaves
// room for scores that grow, and n keys below 2^-14 of fp16's normal range lose at most n 2^-29 of the largest weight.)
template <int D, int NG, typename Settle>
__device__ __forceinline__ void softmax_part(uint32_t (&r)[2][32], uint32_t tC, uint32_t tP, uint32_t tO, const float* sc,
                                             float cs, int visible, bool full, bool first, RowSums& s, Settle settle) {
    constexpr int GK = 64 / NG;
    uint32_t pk[32];
    auto at = [&](int k) { return __uint_as_float(r[k >> 5][k & 31]); };
    auto mask = [&]() {
        if (!full) {
#pragma unroll
            for (int k = 0; k < 64; ++k)
                if (k >= visible) r[k >> 5][k & 31] = 0xff800000u;  // -inf
        }
    };
    // p' of page g, with exponents s ks + b; returns their sum
    auto weigh = [&](int g, float ks, float b) {
        const float2 a2 = make_float2(ks, ks), b2 = make_float2(b, b);
        float2 s0 = make_float2(0.f, 0.f), s1 = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < GK; e += 4) {
            const int k = g * GK + e;
            const float2 y0 = tc::fma2(make_float2(at(k), at(k + 1)), a2, b2), y1 = tc::fma2(make_float2(at(k + 2), at(k + 3)), a2, b2);
            const float2 p0 = make_float2(ex2f(y0.x), ex2f(y0.y)), p1 = make_float2(ex2f(y1.x), ex2f(y1.y));
            s0 = tc::add2(s0, p0);
            s1 = tc::add2(s1, p1);
            pk[k >> 1] = pack_h2(p0.x, p0.y);
            pk[(k >> 1) + 1] = pack_h2(p1.x, p1.y);
        }
        return s0.x + s1.x + (s0.y + s1.y);
    };
    float sum = 0.f;
    bool again = first;
    if (!first) {
        mask();
        const float m_was = s.m == -INFINITY ? 0.f : s.m, mo_was = s.mo == -INFINITY ? 0.f : s.mo;
        float all = 0.f, low = INFINITY;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const float b = sc[8 + g * (GK / 16)] - mo_was, shift = b + m_was;
            low = fminf(low, shift);
            const float part = weigh(g, at_least(cs * sc[g * (GK / 16)]), b);
            all += part;
            sum = fmaf(part, ex2f(-shift), sum);
        }
        again = __any_sync(0xffffffffu, all > 32768.f || low < -60.f || (s.mo == -INFINITY && visible > 0));
    }
    if (!again) {
        tc::tmem_st32(tP, pk);
    } else {
        tc::tmem_ld32(tC, r[0]);
        tc::tmem_ld32(tC + 32, r[1]);
        tc::tmem_ld_wait();
        mask();
        float mx = -INFINITY, mxo = -INFINITY;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            float c0 = -INFINITY, c1 = -INFINITY;
#pragma unroll
            for (int e = 0; e < GK; e += 4) {
                const int k = g * GK + e;
                c0 = tc::fmax3(c0, at(k), at(k + 1));
                c1 = tc::fmax3(c1, at(k + 2), at(k + 3));
            }
            const float y = fmaxf(c0, c1) * at_least(cs * sc[g * (GK / 16)]);
            mx = fmaxf(mx, y);
            mxo = fmaxf(mxo, y + sc[8 + g * (GK / 16)]);
        }
        if (mx > s.m) {
            s.l *= ex2f(s.m - mx);
            s.m = mx;
        }
        const bool move = mxo > s.mo + 8.f;
        float alpha = 1.f;
        if (move) {
            const float to = ceilf(mxo) - 4.f;  // whole numbers, so that rescaling loses nothing
            alpha = ex2f(s.mo - to);
            s.mo = to;
        }
        const float m_use = s.m == -INFINITY ? 0.f : s.m, mo_use = s.mo == -INFINITY ? 0.f : s.mo;
        sum = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const float ks = at_least(cs * sc[g * (GK / 16)]), b = sc[8 + g * (GK / 16)] - mo_use, shift = b + m_use;
            if (__any_sync(0xffffffffu, shift < -60.f)) {
#pragma unroll
                for (int e = 0; e < GK; ++e) sum += ex2f(fmaf(at(g * GK + e), ks, -m_use));
                weigh(g, ks, b);
            } else {
                sum = fmaf(weigh(g, ks, b), ex2f(-shift), sum);
            }
        }
        tc::tmem_st32(tP, pk);
        if (__any_sync(0xffffffffu, move)) {  // last: the wait for the products in flight comes late
            settle(alpha);
            if (!first)
#pragma unroll
                for (int q = 0; q < D / 64; ++q) {
                    uint32_t o[2][32];
                    tc::tmem_ld32(tO + 64 * q, o[0]);
                    tc::tmem_ld32(tO + 64 * q + 32, o[1]);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 64; ++e) o[e >> 5][e & 31] = __float_as_uint(__uint_as_float(o[e >> 5][e & 31]) * alpha);
                    tc::tmem_st32(tO + 64 * q, o[0]);
                    tc::tmem_st32(tO + 64 * q + 32, o[1]);
                }
        }
    }
    s.l += sum;
}

// Where the results of a unit's flat rows go.
struct Out {
    float* slot;  // partial: the share's slot (nullptr: the rows are complete)
    int slot_r;   // its rows
};

// Writes 32 columns (from 32 q on) of flat row m: into the slot; as fp32 to o; or as bf16 into the staging tile at
// `stage`, whose row `row` is this one.
template <int D>
__device__ __forceinline__ void put_cols(const CacheAttnArgs& a, const Seg& g, const Out& out, int m, int row, uint32_t stage,
                                         int q, const float (&v)[32]) {
    if (out.slot) {
        if (m < g.last) {
            float4* dst = reinterpret_cast<float4*>(out.slot) + (8 * q) * out.slot_r + (m - g.m0);
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e * out.slot_r] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
    } else if (a.o_f32) {
        if (m < g.last) {
            float4* dst = reinterpret_cast<float4*>(a.o_f32 + ((long long)(g.row0 + m / a.G) * a.H + g.h * a.G + m % a.G) * D + 32 * q);
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            sts16(stage + row * 2 * D + (((4 * q + e) ^ (row & 7)) << 4), pack_bf2(v[8 * e], v[8 * e + 1]),
                  pack_bf2(v[8 * e + 2], v[8 * e + 3]), pack_bf2(v[8 * e + 4], v[8 * e + 5]), pack_bf2(v[8 * e + 6], v[8 * e + 7]));
    }
}

// Copies rows m_from .. of the staging tile to o, by THREADS threads of which this is number `id`: whole rows, so that
// the stores of a warp are runs of 2 D bytes.
template <int D, int THREADS>
__device__ __forceinline__ void put_rows(const CacheAttnArgs& a, const Seg& g, int m_from, uint32_t stage, int id) {
    constexpr int PER = D / 8, ROWS = THREADS / PER;
    const int chunk = id % PER, dr = ROWS / a.G, dm = ROWS - dr * a.G;
    int r = id / PER, row = (m_from + r) / a.G, rem = m_from + r - row * a.G;
    const int n = imin(128, g.last - m_from);
    __nv_bfloat16* o = a.o + ((long long)g.row0 * a.H + g.h * a.G) * D + 8 * chunk;
#pragma unroll 4
    for (; r < n; r += ROWS) {
        uint32_t v[4];
        lds16(stage + r * 2 * D + ((chunk ^ (r & 7)) << 4), v);
        *reinterpret_cast<uint4*>(o + ((long long)row * a.H + rem) * D) = make_uint4(v[0], v[1], v[2], v[3]);
        row += dr;
        rem += dm;
        if (rem >= a.G) {
            rem -= a.G;
            ++row;
        }
    }
}

__device__ __forceinline__ void put_lse(const CacheAttnArgs& a, const Seg& g, const Out& out, int D, int m, float l2) {
    if (m >= g.last) return;
    if (out.slot) {
        out.slot[(long long)out.slot_r * D + m - g.m0] = l2;
    } else {
        const int row = m / a.G;
        a.lse[(long long)(g.h * a.G + m - row * a.G) * a.total_rows + g.row0 + row] = l2 * 0.69314718055994531f;
    }
}

template <int D, int NG>
__device__ __forceinline__ void softmax(const Ctx<D>& x, const CacheAttnArgs& a, const Start& st) {
    using L = Smem<D>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tS = x.tmem + lane_base, tO = x.tmem + 256 + lane_base;
    const float* scales = reinterpret_cast<const float*>(g_smem + L::kScale);
    Place* place = x.place();
    begin_share(a, st, place);
    uint32_t t = 0, seg = 0, s0_phases = 0;  // s0_phases: bit of each B_S0 stage's next phase
    bool ok = true;  // warp-uniform; once it is false the loops run on without waiting, through the same barriers
    auto wait = [&](int base, int n, uint32_t parity) {
        if (ok) ok = __all_sync(0xffffffffu, x.wait(base, n, parity));
        tc::tc_fence_after();
    };
    while (next_run(a, place)) {
        const int nt = place->g.tiles();
        const bool two = place->g.two;
        float cs;
        int sees, all_see;
        bool warp_live;
        {
            const Seg g = place->g;
            const int m = g.m0 + (two ? 128 * i : 0) + row;  // this thread's flat row
            if (nt == 0) {                                   // rows without keys
                if (m < g.last && (two || i == 0)) {
                    const long long at = ((long long)(g.row0 + m / a.G) * a.H + g.h * a.G + m % a.G) * D;
                    for (int c = 0; c < D; c += 8) {
                        if (a.o_f32) {
                            *reinterpret_cast<float4*>(a.o_f32 + at + c) = make_float4(0.f, 0.f, 0.f, 0.f);
                            *reinterpret_cast<float4*>(a.o_f32 + at + c + 4) = make_float4(0.f, 0.f, 0.f, 0.f);
                        } else {
                            *reinterpret_cast<uint4*>(a.o + at + c) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    put_lse(a, g, Out{nullptr, 0}, D, m, -INFINITY);
                }
                continue;
            }
            split_q<D>(x, a, g);
            tc::fence_proxy_async_smem();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(x.bar(B_Q, 0));
            softmax_sync();  // the rows' exponents
            // the factor that turns the tensor core's q . k8 into base-2 scores; a row that is not finite becomes NaN, and
            // no other
            const int qe = g_smem[L::kQExp + (two ? 128 * i : 0) + row];
            cs = qe == 255 ? NAN : a.scale_log2 * __uint_as_float((uint32_t)qe << 23);
            const int end = m < g.last ? key_end(g.len, a.block, g.pos0 + m / a.G) : 0;
            warp_live = __shfl_sync(0xffffffffu, (int)(m < g.last), 0);
            // keys of a tile that this row sees of the thread's part, and that the warp's first row (which sees the
            // fewest) does
            sees = end - g.kt0 * kTileKeys - (two ? 0 : 64 * i);
            all_see = __shfl_sync(0xffffffffu, sees, 0);
        }
        RowSums sums{-INFINITY, -INFINITY, 0.f};
        uint32_t stage = t % kStages, ph = (t / kStages) & 1, slot = t % kScaleSlots;
        auto up = [&]() {
            sees -= kTileKeys;
            all_see -= kTileKeys;
            slot = slot + 1 == kScaleSlots ? 0 : slot + 1;
            if (++stage == kStages) {
                stage = 0;
                ph ^= 1;
            }
        };
        auto pass_on = [&](int n) {  // p' is in TMEM
            tc::tmem_st_wait();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(x.bar(B_P, n));
        };
        constexpr int NGP = NG > 1 ? NG / 2 : 1;  // pages in 64 keys
        if (two) {
#pragma unroll 1
            for (int j = 0; j < nt; ++j, ++t) {
                if (i == 0) {
                    wait(B_S0, stage, (s0_phases >> stage) & 1);
                } else {
                    wait(B_S1, stage, ph);
                }
                if (warp_live) {
                    uint32_t r[2][32];
                    const uint32_t tC = tS + 128 * i;
                    const float* sc = scales + 16 * slot;
                    tc::tmem_ld32(tC, r[0]);
                    tc::tmem_ld32(tC + 32, r[1]);
                    tc::tmem_ld_wait();
                    // S of a tile is issued behind the PV of the one before, so O is settled
                    softmax_part<D, NGP>(r, tC, tC, tO + D * i, sc, cs, sees, all_see >= 64, j == 0, sums, [](float) {});
                    tc::tmem_ld32(tC + 64, r[0]);
                    tc::tmem_ld32(tC + 96, r[1]);
                    tc::tmem_ld_wait();
                    softmax_part<D, NGP>(r, tC + 64, tC + 32, tO + D * i, sc + 4, cs, sees - 64, all_see >= 128, j == 0, sums, [&](float alpha) {
                        // What the first half has stored. p' is up to 2^15, so an alpha below 2^-24, where fp16 ends,
                        // leaves some of it: two factors, of which the first rounds only what ends below 2^-24.
                        uint32_t w[32];
                        tc::tmem_st_wait();
                        tc::tmem_ld32(tC, w);
                        tc::tmem_ld_wait();
                        const bool far = alpha < 0x1p-15f;
                        const __half2 f0 = __float2half2_rn(far ? 0x1p-15f : alpha), f1 = __float2half2_rn(far ? alpha * 0x1p15f : 1.f);
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const __half2 y = __hmul2(__hmul2(*reinterpret_cast<const __half2*>(&w[e]), f0), f1);
                            w[e] = *reinterpret_cast<const uint32_t*>(&y);
                        }
                        tc::tmem_st32(tC, w);
                    });
                }
                pass_on(2 * (t & 1) + i);
                s0_phases ^= 1u << stage;
                up();
            }
        } else {
#pragma unroll 1
            for (int j = 0; j < nt; ++j, ++t) {
                wait(B_S1, stage, ph);
                if (warp_live) {
                    uint32_t r[2][32];
                    const uint32_t tC = tS + 128 * (t & 1) + 64 * i;
                    tc::tmem_ld32(tC, r[0]);
                    tc::tmem_ld32(tC + 32, r[1]);
                    tc::tmem_ld_wait();
                    softmax_part<D, NGP>(r, tC, tC, tO + D * i, scales + 16 * slot + 4 * i, cs, sees, all_see >= 64, j == 0, sums, [&](float) {
                        if (j > 0) wait(B_PV, (t - 1) & 1, ((t - 1) >> 1) & 1);
                    });
                }
                pass_on(2 * (t & 1) + i);
                up();
            }
        }
        wait(B_PV, (t - 1) & 1, ((t - 1) >> 1) & 1);  // every product of the unit is done
        const Seg g = place->g;
        const int m = g.m0 + (two ? 128 * i : 0) + row, end = m < g.last ? key_end(g.len, a.block, g.pos0 + m / a.G) : 0;
        Out out;
        out.slot_r = slot_rows(a.total_rows, a.G);
        out.slot = g.whole ? nullptr : slot_at(a.scratch, 2 * (int)blockIdx.x + (g.kt0 > 0 ? 0 : 1), out.slot_r, D);
        int* nan_first = reinterpret_cast<int*>(g_smem + L::kNan) + (seg & 3) * D;
        int* nan_any = reinterpret_cast<int*>(g_smem + L::kNanAny) + (seg & 3);
        ++seg;
        const bool staged = !out.slot && !a.o_f32;
        const bool nans = *nan_any < g.end;
        float mj = sums.m, lj = sums.l, f0, f1 = 0.f;
        bool use0 = sums.l != 0.f, use1 = false;  // NaN counts as something
        // o = sum of O_i 2^(mo_i - m) / l over the row's O; one without keys that the row sees adds nothing
        if (two) {
            f0 = use0 ? ex2f(sums.mo - mj) / lj : 0.f;
        } else {
            // the groups exchange their sums through S columns (same lanes); f0 is the own O's factor, f1 the other's
            tmem_st4(tS + 128 * i, __float_as_uint(sums.m), __float_as_uint(sums.mo), __float_as_uint(sums.l), 0u);
            tc::tmem_st_wait();
            tc::tc_fence_before();
            softmax_sync();
            tc::tc_fence_after();
            uint32_t y[4];
            tmem_ld4(tS + 128 * (i ^ 1), y);
            tc::tmem_ld_wait();
            const float m1 = __uint_as_float(y[0]), l1 = __uint_as_float(y[2]);
            use1 = l1 != 0.f;
            mj = fmaxf(sums.m, m1);
            lj = 0.f;
            if (use0) lj += sums.m == mj ? sums.l : sums.l * ex2f(sums.m - mj);
            if (use1) lj += m1 == mj ? l1 : l1 * ex2f(m1 - mj);
            const float inv = 1.f / lj;  // used only where lj is not 0
            f0 = use0 ? ex2f(sums.mo - mj) * inv : 0.f;
            f1 = use1 ? ex2f(__uint_as_float(y[1]) - mj) * inv : 0.f;
        }
        // The S products no longer need Q: the rows of tile i take the place of Q tile i (a unit of one tile: the second)
        const uint32_t tile = x.base + L::kQ + (two ? i : 1) * 2 * L::kT8;
        if (warp_live) {
            const int n = two ? D / 32 : D / 64;
#pragma unroll 1
            for (int k = 0; k < n; ++k) {
                const int q = two ? k : i * n + k;
                uint32_t o[32], o1[32];
                tc::tmem_ld32(tO + D * i + 32 * q, o);
                if (!two) tc::tmem_ld32(tO + D * (i ^ 1) + 32 * q, o1);
                tc::tmem_ld_wait();
                float v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    v[e] = (use0 ? __uint_as_float(o[e]) * f0 : 0.f) + (use1 ? __uint_as_float(o1[e]) * f1 : 0.f);
                if (nans)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (nan_first[32 * q + e] < end) v[e] = NAN;
                put_cols<D>(a, g, out, m, row, tile, q, v);
            }
        }
        if (two || i == 0) put_lse(a, g, out, D, m, lj != 0.f ? mj + __log2f(lj) : -INFINITY);
        tc::tc_fence_before();
        if (staged) {
            if (two) {
                group_sync(i);
                put_rows<D, 128>(a, g, g.m0 + 128 * i, tile, row);
            } else {
                softmax_sync();
                put_rows<D, 256>(a, g, g.m0, tile, threadIdx.x);
            }
        }
        // The next unit's Q may be written once both groups are done with this one. The widening warps are at most two
        // tiles ahead of the PV products, so they come back to these words only after three more units have begun.
        softmax_sync();
        if (nans && threadIdx.x < D) nan_first[threadIdx.x] = *nan_any = 0x7fffffff;
    }
}

// ------------------------------------------------------------------- kernel
template <int D, int NG>
__global__ void __launch_bounds__(kThreads, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const CacheAttnArgs a) {
    using L = Smem<D>;
    Ctx<D> x;
    x.base = sbase();
    Start* st = reinterpret_cast<Start*>(g_smem + L::kStart);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = tid; i < 4 * D + 4; i += kThreads) reinterpret_cast<int*>(g_smem + L::kNan)[i] = 0x7fffffff;
    if (tid == 0) {
        x.words()[1] = x.words()[2] = 0;
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(x.bar(B_KFULL, s), 1);
            tc::mbar_init(x.bar(B_S0, s), 1);
            tc::mbar_init(x.bar(B_S1, s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(x.bar(B_VFULL, s), 1);
            tc::mbar_init(x.bar(B_VEMPTY, s), 4);  // lane 0 of the widening warps
            tc::mbar_init(x.bar(B_P, 2 * s), kSoftmax / 64 + 4);  // lane 0 of group 0's warps and of the widening warps
            tc::mbar_init(x.bar(B_P, 2 * s + 1), kSoftmax / 64);
            tc::mbar_init(x.bar(B_PV, s), 1);
        }
        tc::mbar_init(x.bar(B_Q, 0), kSoftmax / 32);
        tc::fence_barrier_init();
    }
    if (warp == 9) {
        tc::tmem_alloc(tc::smem_addr(x.words()), kTmemCols);
        tc::tmem_relinquish();
    }
    if (warp == 8 && lane == 0) {
        tc::prefetch_tmap(&tk);
        tc::prefetch_tmap(&tv);
    }
    find_start(a, st, reinterpret_cast<long long*>(g_smem));  // the scan's words lie where Q will
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    x.tmem = (uint32_t)x.words()[0];
    // the swizzled tiles need the one, the MMA warp counts on the other; a launch that has not is refused
    const bool aligned = (sbase() & 1023u) == 0 && x.tmem == 0;
    if (tid == 0 && !aligned) x.words()[1] = 1;
    if (st->left > 0 && aligned) {
        if (warp >= 8) {
            tc::regs_dec<kRegsOther>();
            if (warp == 8) produce<D>(x.own(), a, *st, &tk, &tv);
            else if (warp == 9) issue<D>(a, *st);
            else if (warp >= 12) widen<D>(x.own(), a, *st);
        } else {
            tc::regs_inc<kRegsSoftmax>();
            softmax<D, NG>(x.own(), a, *st);
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
        r.per = st->per;
        r.more = st->more;
        r.C = st->C;
        if (st->left > 0) {
            const SeqRows q = seq_rows(a.c, a.cu_rows, a.q_pos, a.total_rows, st->s);
            r.row0 = q.row0;
            r.rows = q.rows;
            r.pos0 = q.pos0;
            r.len = q.len;
            r.head = st->h;
            r.m0 = st->m0;
            r.off = st->off;
            r.cost = unit_of(a, q, st->m0).cost();
        }
        r.error = x.words()[1] ? DEV_TIMEOUT : st->bad != 0x7fffffff ? DEV_CHECK : x.words()[2];
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
