// What the kernels of attention with many q rows share: the walk over a CTA's units, and where its results go.
#pragma once

#include <math_constants.h>

#include "paged_common.cuh"
#include "ptx_sync.cuh"

namespace qkv_rows {

using namespace qkv_paged;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Units of a CTA, the last ones' fewer.  (A least share, for a part costs its write and its join, of 3 units made 17 new tokens
// 21.5 us instead of 19.5, one of 6 units 20 sequences on a prefix 67 instead of 60, and nothing faster.)
__device__ __forceinline__ int64_t share_of(int64_t total, int ctas) { return (total + ctas - 1) / ctas; }

// What a tile counts for in the sharing out besides its blocks: its beginning and end, for either half of its rows.
__device__ __forceinline__ int tile_cost(const PagedRowsParams& p, const RowTile& t) {
    return t.ntok > p.part_tokens ? 2 * p.tile_cost : p.tile_cost;
}

// Some units [from, to) of one tile, and the first q head.
struct Piece {
    RowTile t;
    int tile, head;  // head: kv head and block of its q heads
    int from, to;
    bool first;      // the tile lies over the CTA's beginning
    bool begin, end, all;  // where pieces are limited: the first, the last of the tile's units in the CTA; these are all it has
};

__device__ __forceinline__ RowTile load_tile(const PagedRowsParams& p, int i) {
    RowTile t;
    const int4* s = reinterpret_cast<const int4*>(p.tiles + i);
    int4* d = reinterpret_cast<int4*>(&t);
    static_assert(sizeof(RowTile) == 48, "three loads");
    d[0] = __ldcg(s);
    d[1] = __ldcg(s + 1);
    d[2] = __ldcg(s + 2);
    return t;
}

// The units of one CTA, piece by piece, of MOST units at most.  Every warp walks for itself; all its lanes call together.
template <int MOST = 0x7fffffff>
struct Walk {
    static constexpr bool kLimited = MOST < 0x7fffffff;
    int64_t at, end, per_head, share;
    int tiles, tile, head;
    // Whether the CTA has all of the tile; and this piece is the last of it.
    static __device__ __forceinline__ bool all(const Piece& x) { return kLimited ? x.all : x.from == 0 && x.to == x.t.units; }
    static __device__ __forceinline__ bool whole(const Piece& x) { return all(x) && (!kLimited || x.end); }
    __device__ __forceinline__ bool begin(const PagedRowsParams& p) {
        per_head = __ldcg(p.total);
        tiles = static_cast<int>(__ldcg(p.total + 1));
        const int64_t total = per_head * p.nkv * p.blocks;
        share = share_of(total, gridDim.x);
        at = share * blockIdx.x;
        end = min(total, at + share);
        if (at >= end) return false;
        head = static_cast<int>(at / per_head);
        const int64_t r = at - head * per_head;
        // the last tile that begins at or before r: 32 candidates at a time
        int lo = 0, n = tiles;
        const int lane = threadIdx.x & 31;
        while (n > 1) {
            const int step = (n + 31) / 32, i = lo + lane * step;
            const bool ok = lane * step < n && __ldcg(&p.tiles[i].start) <= r;
            const int last = 31 - __clz(__ballot_sync(0xffffffffu, ok));
            lo += last * step;
            n = min(step, n - last * step);
        }
        tile = lo;
        return true;
    }
    __device__ __forceinline__ bool next(const PagedRowsParams& p, Piece& x) {
        while (at < end) {
            if (tile >= tiles) {
                tile = 0;
                ++head;
            }
            x.t = load_tile(p, tile);
            const int64_t start = head * per_head + x.t.start;
            x.tile = tile++;
            if (x.t.units == 0) continue;
            x.head = head;
            const int stop = static_cast<int>(min(static_cast<int64_t>(x.t.units), end - start));
            x.from = static_cast<int>(min(at - start, static_cast<int64_t>(x.t.units)));
            x.to = kLimited && stop - x.from > MOST ? x.from + MOST : stop;
            x.first = start <= share * blockIdx.x;
            if (kLimited) {
                x.begin = at == max(start, share * blockIdx.x);
                x.end = x.to == stop;
                x.all = start >= share * blockIdx.x && stop == x.t.units;
                if (!x.end) {  // the same tile again
                    at = start + x.to;
                    --tile;
                    return true;
                }
            }
            at = start + x.t.units + tile_cost(p, x.t);
            if (x.from < x.to) return true;  // else only the tile's end is this CTA's
        }
        return false;
    }
};

// Row of a tile for its token i and q head g of the block.
__device__ __forceinline__ int row_of(const PagedRowsParams& p, int i, int g) {
    const int part = i / p.part_tokens;
    return part * p.part_rows + (i - part * p.part_tokens) * p.per_block + g;
}

// What row i of a tile sees.
__device__ __forceinline__ void row_span(const PagedRowsParams& p, const RowTile& t, int i, int& lo, int& hi) {
    if (p.first) {
        hi = max(0, t.base + i);
        lo = p.window > 0 ? max(0, t.base + i - p.window) : 0;
    } else {
        hi = __ldcg(p.row_end + t.row0 + i);
        lo = 0;
    }
}

__device__ __forceinline__ float* part_of(const PagedRowsParams& p, int cta, bool first) {
    return p.part + static_cast<int64_t>(2 * cta + (first ? 0 : 1)) * p.rows * (p.hd + 2);
}
// Maximum and sum of a part's row; the rows' sums of V come behind all of these.
__device__ __forceinline__ float2* part_ml(float* part, int row) { return reinterpret_cast<float2*>(part) + row; }
__device__ __forceinline__ float* part_o(const PagedRowsParams& p, float* part, int row) {
    return part + 2 * p.rows + static_cast<int64_t>(row) * p.hd;
}

// For the join: the CTA in which a tile begins notes how many CTAs have parts of it; one thread, first for no piece.
__device__ __forceinline__ void note_none(const PagedRowsParams& p) { p.pieces[blockIdx.x].parts = 0; }
template <typename W>
__device__ __forceinline__ void note_piece(const PagedRowsParams& p, const W& w, const Piece& x) {
    if (x.from > 0 || w.all(x)) return;
    RowPiece r = {};
    r.start = x.head * w.per_head + x.t.start;
    r.tile = x.tile;
    r.head = x.head;
    r.parts = static_cast<int>((r.start + x.t.units - 1) / w.share - blockIdx.x) + 1;
    p.pieces[blockIdx.x] = r;
}

__device__ __forceinline__ uint16_t bf16_bits(float v) {
    uint16_t r;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ void put_out(const PagedRowsParams& p, int64_t at, float v) {
    if (p.out_bf16) static_cast<uint16_t*>(p.out)[at] = bf16_bits(v);
    else static_cast<float*>(p.out)[at] = v;
}
// log(l 2^m); an empty row has none.
__device__ __forceinline__ float lse_of(float m, float l, bool empty) {
    return empty ? -CUDART_INF_F : (m + log2f(l)) * kLn2;
}

}  // namespace qkv_rows
