// cache_attn.cuh - what the attention kernel over the paged cache and the merge
// of its partial results share: how the work is cut, and where partials lie.
//
// A unit is (sequence, kv head, run of 256 flat rows): the rows r * G + g of a
// sequence's new rows r and of the G query heads g that share the kv head,
// which all read the same keys. Its tiles are its runs of 128 keys, up to the
// last key that its last row sees (one, without keys, if it sees none). Its
// cost is its tiles and a lead for what it takes to begin and to end it (query,
// results), twice that for a unit of two MMA tiles. All units'
// costs, laid end to end (sequence, head, run), are cut into equal shares, one
// per CTA (the first W % C of them one longer). A share that begins or ends
// between the tiles of a unit leaves a partial result; at most two per CTA,
// slot 2 c for a unit begun by an earlier CTA and slot 2 c + 1 for one that a
// later CTA goes on with.
//
// With runs (a.runs) the same is done over items instead of sequences. Item
// 2 s is the pages that a run led by sequence s shares, read by the rows of
// all of the run's sequences (they lie side by side) as if they were one
// sequence's; item 2 s + 1 is what sequence s reads alone. Rows of a run get
// two partial results, one of each kind, in two planes, which are joined at the
// end. A plane holds flat rows, of each kv head, as a slot holds a unit's, so
// units of either kind may be cut anywhere: all of the call's, or, where those
// are more, 128 for each sequence. A run that is read together has fewer than
// that for each of its sequences with rows, and its rows lie side by side from
// the place of its first sequence on (69500 rows of 32 heads in 16 sequences,
// d = 128: 34 MB instead of 2.3 GB).
#pragma once

#include "cache.cuh"

namespace bdlm {
namespace cattn {

constexpr int kTileKeys = 128;
constexpr int kUnitRows = 256;
constexpr int kMaxCtas = 256;
// What beginning and ending a unit costs, in tiles of 128 keys, besides a tile for every 32 rows of an MMA tile that is
// alive (lead_of). Measured with 3, 4, 5, 6: 64 sequences of one row (4 flat rows per unit, 512 to 30912 keys) 230, 219,
// 212, 210 us; 37 ragged ones (1 to 47 rows, up to 9001 keys) 37.6, 38.3, 38.6, 40.2 us. Without the tiles for the rows,
// 64 sequences of 32 rows (128 flat rows per unit) took 251 instead of 235 us.
constexpr int kLead = 5;
// A share is at least this long where there is too little work for all CTAs: below it the partial results cost more
// than the shorter shares save. One row over 600 keys takes 15.3, 16.0, 16.8, 18.3 us with 2, 3, 4, 6; three rows over
// 56 to 277 keys 17.9, 17.6, 17.7, 16.3. (At least 2, so that each of the shares of a unit holds a tile of it.)
constexpr int kMinShare = 3;

// What CTA c leaves for the merge: where its share begins, and its errors.
struct ShareRec {
    int row0, rows, pos0, len;  // the sequence (SeqRows) whose unit the share begins in; row0 of rows in a plane: Rows::plane
    int head, m0;               // kv head and first flat row of that unit
    int off, cost;              // where in the unit's cost the share begins, the unit's cost
    long long per;              // share_begin's constants
    int more, C;                // C: shares
    int error, info;
    int part;  // of the unit: Rows::part
    int bad;   // malformed arguments: nothing was computed
};
static_assert(sizeof(ShareRec) == 64, "share record is 64 bytes");

__host__ __device__ __forceinline__ int slot_rows(long long total_rows, int G) {
    const long long flat = total_rows * G;
    return flat >= kUnitRows ? kUnitRows : (int)((flat + 7) / 8 * 8);
}
// With runs a unit is one MMA tile: what is read together is seldom long enough for units of two to pay for their longer
// beginnings and ends (64 single rows over 32768 shared keys: 93 us whole with two, 66 with one).
template <bool RUNS>
__host__ __device__ constexpr int unit_rows() { return RUNS ? kUnitRows / 2 : kUnitRows; }

// A slot: normalised fp32 rows as [D / 4][rows] float4 (a warp's rows are
// consecutive), then the rows' base-2 lse.
__host__ __device__ __forceinline__ long long slot_floats(int rows, int D) { return (long long)rows * (D + 1) + (32 - rows % 32) % 32; }

__device__ __forceinline__ ShareRec* share_recs(uint8_t* scratch) { return reinterpret_cast<ShareRec*>(scratch); }
__device__ __forceinline__ float* slot_at(uint8_t* scratch, int slot, int rows, int D) {
    return reinterpret_cast<float*>(scratch + sizeof(ShareRec) * kMaxCtas) + slot * slot_floats(rows, D);
}

// Where share c of C begins; per = W / C, more = W % C.
__device__ __forceinline__ long long share_begin(long long per, int more, int c) { return per * c + imin(c, more); }

// The rows of an item, and the keys that they read: those of `seq` at
// positions [key0, len) that each row sees.
struct Rows : SeqRows {
    int seq;
    int key0;
    int part;  // where results go: 0 to o and lse, 1 and 2 into the first and second plane
    int plane;  // there: the first flat row's place
};
enum : int { PART_WHOLE = 0, PART_SHARED = 1, PART_OWN = 2 };

// Sequences with few flat rows and few keys of their own (`own`: those behind what they share) do not pay for an MMA tile:
// cache_own_kernel reads those keys, one CTA for a sequence's head. One row each of n sequences over 8192 shared keys and 256,
// 1024, 2048, 4096 own ones (8 kv heads, d = 128, G = 4), us by tiles: 33, 32, 35, 36 for n = 4, 71, 97, 127, 179 for 64, 205,
// 287, 397, 610 for 256; by that kernel 34, 34, 36, 49, then 49, 75, 97, 140, and 125, 178, 252, 401. So the longest
// are left to it where there are CTAs enough to fill the SMs.
constexpr int kFewRows = 8, kFewKeys = 2048, kMostKeys = 4096, kManyCtas = 256;
__device__ __forceinline__ int few_keys(const CacheAttnArgs& a) { return a.c.n_seqs * a.c.Hk >= kManyCtas ? kMostKeys : kFewKeys; }
__device__ __forceinline__ bool is_few(const CacheAttnArgs& a, int rows, int own) { return rows * (long long)a.G <= kFewRows && own <= few_keys(a); }

// Whether n sequences with rows, `rows` in all, gain from reading `shared` positions together, in keys of a tile's time. Alone,
// each takes MMA tiles of 128 flat rows through them, however few it has, or, if those are few, cache_own_kernel, in which a
// key takes four fifths of that; together they take what their rows fill (those that fill a tile each gain nothing). Against
// that stand, in tiles, the units that this adds and the joins, kRowCost for a flat row, or, where rows are few, kOwnCost for a
// sequence; and 32 for the call (a.call_tiles for each of the sequences that may have rows), if nothing else in it is read together. Twice as
// many tiles of d = 64, which take half the time.
// Alone and together, us, with 1024 shared keys (d = 128, G = 4, 100 own keys): 64 sequences of 1 row 38, 33; 16 runs of 4 38,
// 45; 16 of 16 116, 85; with 8 rows each 100, 71; 97, 76; 361, 244; a run of 8 with 8 rows 31, 32; with 16 rows 16 runs of 4 105,
// 108; 16 of 16 358, 345. (Without contractions: every kernel must come to the same.)
constexpr float kRowCost = 0.053f, kOwnCost = 4.f;
constexpr int kPlaneRows = 128;  // an MMA tile's
static_assert(kFewRows < kPlaneRows, "rows of a run have places in the planes");
__device__ __forceinline__ bool worth(const CacheAttnArgs& a, int n, int rows, int shared) {
    const int flat = rows * a.G, together = (flat + 127) >> 7;
    const float wide = a.c.D == 128 ? (float)kTileKeys : 2.f * kTileKeys;
    if (flat <= kFewRows * n && shared <= few_keys(a))
        return __fmul_rn((float)shared, (float)(4 * n - 5 * together)) > __fmul_rn(__fmul_rn(5.f * wide, (float)n), __fadd_rn(kOwnCost, a.call_tiles));
    return flat < kPlaneRows * n && __fmul_rn((float)shared, (float)(n - together)) >
                                 __fmul_rn(wide, __fadd_rn(__fmul_rn(kRowCost, (float)flat), __fmul_rn((float)n, a.call_tiles)));
}

// Those without rows among a run's sequences read nothing and are not joined, so they do not count. A whole warp counts the
// others: for all of its lanes at once where they name the SAME run, else for one run after the other, of which `last` is
// kept. Short ones a lane counts by itself.
struct Busy {
    int first = -1, end = -1, n = 0;
};
__device__ __forceinline__ int busy_in(const CacheAttnArgs& a, int first, int end) {
    int n = 0;
    for (int i0 = first; i0 < end; i0 += 32) {
        const int i = i0 + (int)(threadIdx.x & 31);
        n += __popc(__ballot_sync(0xffffffffu, i < end && __ldg(a.cu_rows + i + 1) > __ldg(a.cu_rows + i)));
    }
    return n;
}
constexpr int kCounted = 128;
template <bool SAME>
__device__ __forceinline__ int busy_of(const CacheAttnArgs& a, int first, int end, bool ask, Busy* last) {
    constexpr int kShort = 8;
    if (SAME) return ask ? busy_in(a, first, end) : 0;
    int n = 0;
    if (ask && end - first <= kShort) {
        int at[kShort + 1];
#pragma unroll
        for (int k = 0; k <= kShort; ++k) at[k] = first + k <= end ? __ldg(a.cu_rows + first + k) : 0;
#pragma unroll
        for (int k = 0; k < kShort; ++k) n += at[k + 1] > at[k];  // (0 is no more than what is before it)
        ask = false;
    }
    for (;;) {
        if (ask && first == last->first && end == last->end) {
            n = last->n;
            ask = false;
        }
        const unsigned todo = __ballot_sync(0xffffffffu, ask);
        if (!todo) return n;
        const int src = __ffs(todo) - 1;
        last->first = __shfl_sync(0xffffffffu, first, src);
        last->end = __shfl_sync(0xffffffffu, end, src);
        last->n = busy_in(a, last->first, last->end);
    }
}

// What the run of sequence s is, and whether it is well-formed: all of its
// sequences name the same one, and share no more than each of their rows sees.
// Called by whole warps.
struct Run {
    int first, end, shared;
    int plane;  // place of the sequence's first flat row in the planes, if it is read together
    bool ok;
};
template <bool CHECK, bool SAME>
__device__ __forceinline__ Run run_of(const CacheAttnArgs& a, int s, const SeqRows& r, Busy* last) {
    const int n = a.c.n_seqs;
    const int *f = a.runs, *e = a.runs + n, *h = a.runs + 2 * (long long)n;
    Run u{__ldg(f + s), __ldg(e + s), __ldg(h + s), 0, true};
    if (CHECK) {  // (else another kernel, or this one's beginning, has looked it over)
        // the neighbours' too at once: loads that wait for one another are what this costs
        const int i = imax(s - 1, 0), j = imin(s + 1, n - 1);
        const bool before = __ldg(f + i) == u.first && __ldg(e + i) == u.end && __ldg(h + i) == u.shared;
        const bool behind = __ldg(f + j) == u.first && __ldg(e + j) == u.end && __ldg(h + j) == u.shared;
        u.ok = u.first >= 0 && u.first <= s && u.end > s && u.end <= n && u.shared >= 0 && (u.shared & (a.c.page - 1)) == 0;
        u.ok = u.ok && (u.first == s || before) && (u.end == s + 1 || behind);
        if (u.shared > 0 && (s == u.first || r.rows > 0)) u.ok = u.ok && u.shared <= r.len && (r.rows == 0 || u.shared <= r.pos0);
    }
    // (a long run that would not gain if all that may have rows had some is not counted)
    const bool asked = u.ok && u.shared > 0;
    const int row0 = asked ? __ldg(a.cu_rows + u.first) : 0;
    const int span = u.end - u.first, rows = asked ? __ldg(a.cu_rows + u.end) - row0 : 0;
    const bool count = asked && (span <= kCounted || worth(a, imin(span, rows), rows, u.shared));
    const int busy = busy_of<SAME>(a, u.first, u.end, count, last);
    if (u.ok && !(count && worth(a, busy, rows, u.shared))) u.shared = 0;
    // (worth: fewer than kPlaneRows flat rows for each that is counted)
    u.plane = a.plane_rows < a.total_rows * a.G ? kPlaneRows * u.first + (r.row0 - row0) * a.G : r.row0 * a.G;
    return u;
}

template <bool RUNS>
__device__ __forceinline__ int items_of(const CacheAttnArgs& a) { return RUNS ? 2 * a.c.n_seqs : a.c.n_seqs; }

// All lanes of a warp ask for the same item, or with `last` each for one of its own.
template <bool RUNS, bool CHECK = false, bool SAME = true>
__device__ __forceinline__ Rows item_rows(const CacheAttnArgs& a, int item, Busy* last = nullptr) {
    Rows r;
    r.seq = RUNS ? item >> 1 : item;
    static_cast<SeqRows&>(r) = seq_rows(a.c, a.cu_rows, a.q_pos, a.total_rows, r.seq);
    r.key0 = 0;
    r.part = PART_WHOLE;
    r.plane = 0;
    if (RUNS) {
        const Run u = run_of<CHECK, SAME>(a, r.seq, r, last);
        r.ok = r.ok && u.ok;
        r.plane = u.plane;
        if (item & 1) {
            if (u.shared > 0) {
                r.key0 = u.shared;
                r.part = PART_OWN;
            }
            if (r.ok && is_few(a, r.rows, r.len - r.key0)) r.rows = 0;
        } else if (!r.ok || u.shared == 0 || u.first != r.seq) {
            r.rows = 0;
        } else {
            const int b = __ldg(a.cu_rows + u.end);
            r.ok = b >= r.row0 && b <= a.total_rows;
            r.rows = r.ok ? b - r.row0 : 0;
            r.len = u.shared;
            r.pos0 = u.shared - 1;  // the first row sees them all, and so do the others
            r.part = PART_SHARED;
        }
    }
    return r;
}

// Keys of its item that the row at position p sees.
template <bool RUNS, typename T>
__device__ __forceinline__ int keys_of(const CacheAttnArgs& a, const T& r, int p) {
    return key_end(r.len, a.block, p) - (RUNS ? r.key0 : 0);
}

// A plane: for each kv head normalised fp32 rows as [D / 4][plane_rows] float4; behind both planes the rows' base-2 lse
// [Hk][plane_rows] twice.
__device__ __forceinline__ float* plane_o(const CacheAttnArgs& a, int D, int part, int head) {
    const long long flat = a.plane_rows;
    return a.planes + ((part - 1) * (long long)a.c.Hk + head) * D * flat;
}
__device__ __forceinline__ float* plane_lse(const CacheAttnArgs& a, int D, int part, int head) {
    const long long flat = a.plane_rows;
    return a.planes + (2LL * a.c.Hk * D + (part - 1) * (long long)a.c.Hk + head) * flat;
}

struct Unit {
    int last;   // last flat row + 1
    int end;    // keys that the last row sees
    int tiles;  // at least 1
    int two;    // 1: two MMA tiles
    int lead;   // what it costs besides, in tiles
    __device__ __forceinline__ int cost() const { return (lead + tiles) << two; }
};
__device__ __forceinline__ int is_two(int rows) { return rows > kUnitRows / 2; }
__device__ __forceinline__ int lead_of(int rows) { return kLead + ((rows + 31) >> (5 + is_two(rows))); }
template <bool RUNS>
__device__ __forceinline__ Unit unit_of(const CacheAttnArgs& a, const Rows& r, int m0) {
    Unit u;
    u.last = imin(r.rows * a.G, m0 + unit_rows<RUNS>());
    u.end = keys_of<RUNS>(a, r, r.pos0 + (u.last - 1) / a.G);
    u.tiles = imax(1, (u.end + kTileKeys - 1) / kTileKeys);
    u.two = RUNS ? 0 : is_two(u.last - m0);
    u.lead = lead_of(u.last - m0);
    return u;
}
// First tile that lies at or behind offset `off` of a unit's cost.
__device__ __forceinline__ int tile_at(int off, int two, int lead) { return imax(0, (off >> two) - lead); }

}  // namespace cattn

cudaError_t launch_cache_attn_d64(const CacheAttnArgs& a, int ctas, cudaStream_t st);
cudaError_t launch_cache_attn_d128(const CacheAttnArgs& a, int ctas, cudaStream_t st);
cudaError_t launch_cache_attn_runs_d64(const CacheAttnArgs& a, int ctas, cudaStream_t st);
cudaError_t launch_cache_attn_runs_d128(const CacheAttnArgs& a, int ctas, cudaStream_t st);

}  // namespace bdlm
