// chunk.cuh -- how the work of chunk attention is laid out, for its kernels: a sequence's new tokens in tiles, a
// tile's visible keys in blocks, and a unit (sequence, KV head, tile) of blocks dealt to CTAs in equal ranges.
#pragma once

#include "kvz_internal.h"

namespace kvz {

constexpr int kChunkBlock = 128;   // keys of a block: 8 pages
constexpr int kChunkRows = 256;    // query rows of a tile: two streams of 128
constexpr int32_t kPageGone = INT32_MIN;  // a page that an earlier kernel of the call has left out and flagged

struct ChunkSeq {
    int q0, n, len, tiles;  // first new token, new tokens, tokens with them, tiles
};

__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkParams &P, int start, int end, int len)
{
    ChunkSeq s;
    s.q0 = start;
    s.n = end - start;
    s.len = named_tokens(len, P.len_pages, P.tail);
    s.tiles = (s.n + P.tile_tokens - 1) / P.tile_tokens;
    return s;
}

// Keys that any token of a tile sees: [lo, hi) and the first `sinks`; in blocks [0, sb) and from wb on.
struct ChunkTile {
    int tokens, p0, lo, hi, sb, wb, blocks;
};

__device__ __forceinline__ ChunkTile chunk_tile(const ChunkParams &P, int n, int len, int k)
{
    ChunkTile t;
    const int t0 = k * P.tile_tokens;
    t.tokens = min(P.tile_tokens, n - t0);
    t.p0 = len - n + t0;
    t.hi = max(0, t.p0 + t.tokens);
    t.lo = P.window > 0 ? max(0, max(t.p0, 0) - P.window + 1) : 0;
    t.wb = t.lo / kChunkBlock;
    const int eb = t.hi / kChunkBlock + (t.hi % kChunkBlock != 0), s = min(P.sinks, t.hi);
    t.sb = min(t.wb, s / kChunkBlock + (s % kChunkBlock != 0));
    t.blocks = max(1, t.sb + eb - t.wb);  // (a tile whose tokens see nothing still has an output)
    return t;
}

// Whether any token of the tile sees a key of the page that begins at key `at`.
__device__ __forceinline__ bool chunk_page_seen(const ChunkParams &P, int lo, int hi, int at)
{
    return at < hi && (at + kPage > lo || at < P.sinks);
}

// Pages that any new token of a sequence sees: [0, sinks) and [first, end).
struct ChunkPages {
    int sinks, first, end;
    __device__ __forceinline__ int count() const { return sinks + end - first; }
    __device__ __forceinline__ int page(int k) const { return k < sinks ? k : first + k - sinks; }
};

__device__ __forceinline__ ChunkPages chunk_pages(const ChunkParams &P, int n, int len)
{
    ChunkPages g;
    const int p0 = len - n, lo = P.window > 0 ? max(0, max(p0, 0) - P.window + 1) : 0, s = min(P.sinks, len);
    g.first = lo / kPage;
    g.end = len / kPage + (len % kPage != 0);
    g.sinks = min(g.first, s / kPage + (s % kPage != 0));
    return g;
}

// First block of CTA c's range of W blocks over C CTAs.
__device__ __forceinline__ int64_t chunk_first(int64_t c, int64_t W, int C) { return (c * W + C - 1) / C; }

}  // namespace kvz
