// cache_attn.cuh - what the attention kernel over the paged cache and the merge
// of its partial results share: how the work is cut, and where partials lie.
//
// A unit is (sequence, kv head, run of 256 flat rows): the rows r * G + g of a
// sequence's new rows r and of the G query heads g that share the kv head,
// which all read the same keys. Its work is its key tiles of 128 keys, up to
// the last key that its last row sees (one, without keys, if it sees none).
// All units' tiles, laid end to end (sequence, head, run, tile), are cut into
// equal shares, one per CTA: CTA c takes the tiles [W c / C, W (c + 1) / C).
// A share that begins or ends inside a unit leaves a partial result; at most
// two per CTA, slot 2 c for a unit begun by an earlier CTA and slot 2 c + 1
// for one that a later CTA goes on with.
#pragma once

#include "cache.cuh"

namespace bdlm {
namespace cattn {

constexpr int kTileKeys = 128;
constexpr int kUnitRows = 256;
constexpr int kMaxCtas = 256;
// A CTA takes at least this many tiles where there are too few for all: below it the partial results cost more than
// the shorter shares save.
constexpr int kMinTiles = 2;

// What CTA c leaves for the merge: where its share begins, and its errors.
struct ShareRec {
    int row0, rows, pos0, len;  // the sequence (SeqRows) whose unit the share begins in
    int head, m0;               // kv head and first flat row of that unit
    int kt0, cost;              // first tile of the share in the unit, tiles of the unit
    long long W;                // tiles of the whole call (0: nothing to do)
    int C;                      // shares
    int error, info;
    int pad[3];
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

__device__ __forceinline__ long long share_begin(long long W, int C, int c) { return W * c / C; }

struct Unit {
    int last;  // last flat row + 1
    int end;   // keys that the last row sees
    int cost;  // tiles, at least 1
};
__device__ __forceinline__ Unit unit_of(const CacheAttnArgs& a, const SeqRows& r, int m0) {
    Unit u;
    u.last = imin(r.rows * a.G, m0 + kUnitRows);
    u.end = key_end(r.len, a.block, r.pos0 + (u.last - 1) / a.G);
    u.cost = imax(1, (u.end + kTileKeys - 1) / kTileKeys);
    return u;
}

}  // namespace cattn

cudaError_t launch_cache_attn_d64(const CacheAttnArgs& a, int ctas, cudaStream_t st);
cudaError_t launch_cache_attn_d128(const CacheAttnArgs& a, int ctas, cudaStream_t st);

}  // namespace bdlm
