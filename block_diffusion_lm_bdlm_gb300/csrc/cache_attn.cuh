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
    int row0, rows, pos0, len;  // the sequence (SeqRows) whose unit the share begins in
    int head, m0;               // kv head and first flat row of that unit
    int off, cost;              // where in the unit's cost the share begins, the unit's cost
    long long per;              // share_begin's constants
    int more, C;                // C: shares
    int error, info;
    int pad[2];
};
static_assert(sizeof(ShareRec) == 64, "share record is 64 bytes");

__host__ __device__ __forceinline__ int slot_rows(long long total_rows, int G) {
    const long long flat = total_rows * G;
    return flat >= kUnitRows ? kUnitRows : (int)((flat + 7) / 8 * 8);
}

// A slot: normalised fp32 rows as [D / 4][rows] float4 (a warp's rows are
// consecutive), then the rows' base-2 lse.
__host__ __device__ __forceinline__ long long slot_floats(int rows, int D) { return (long long)rows * (D + 1) + (32 - rows % 32) % 32; }

__device__ __forceinline__ ShareRec* share_recs(uint8_t* scratch) { return reinterpret_cast<ShareRec*>(scratch); }
__device__ __forceinline__ float* slot_at(uint8_t* scratch, int slot, int rows, int D) {
    return reinterpret_cast<float*>(scratch + sizeof(ShareRec) * kMaxCtas) + slot * slot_floats(rows, D);
}

// Where share c of C begins; per = W / C, more = W % C.
__device__ __forceinline__ long long share_begin(long long per, int more, int c) { return per * c + imin(c, more); }

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
__device__ __forceinline__ Unit unit_of(const CacheAttnArgs& a, const SeqRows& r, int m0) {
    Unit u;
    u.last = imin(r.rows * a.G, m0 + kUnitRows);
    u.end = key_end(r.len, a.block, r.pos0 + (u.last - 1) / a.G);
    u.tiles = imax(1, (u.end + kTileKeys - 1) / kTileKeys);
    u.two = is_two(u.last - m0);
    u.lead = lead_of(u.last - m0);
    return u;
}
// First tile that lies at or behind offset `off` of a unit's cost.
__device__ __forceinline__ int tile_at(int off, int two, int lead) { return imax(0, (off >> two) - lead); }

}  // namespace cattn

cudaError_t launch_cache_attn_d64(const CacheAttnArgs& a, int ctas, cudaStream_t st);
cudaError_t launch_cache_attn_d128(const CacheAttnArgs& a, int ctas, cudaStream_t st);

}  // namespace bdlm
