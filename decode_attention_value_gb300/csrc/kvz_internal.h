// kvz_internal.h -- parameter blocks and launchers shared by the host runtime
// (kvz_api.cu) and the kernels (codec.cu, attention.cu).  Not installed.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kvz_device.cuh"

namespace kvz {

struct EncodeParams {
    int hkv;
    int n;
    const uint16_t *raw_pool;
    int64_t num_raw_pages;
    const int32_t *src_page, *dst_page, *dst_seq;
    uint64_t *meta;
    int64_t num_meta_pages;
    uint8_t *arena;
    uint64_t arena_bytes;
    uint32_t *cursors;
    int num_cursors;
    uint32_t *status;
    // group-adaptive tiles: 4-byte entries instead of meta, bases [hkv][2][2][128]
    uint32_t *meta32;
    const uint8_t *ga_bases;
    // workspace
    uint32_t *ws_hdr;        // [4]: validation failure bits (stored by the prepare kernel each call)
    uint32_t *ws_page_size;  // [n] granules per page, summed over heads (zeroed each call)
    uint32_t *ws_page_base;  // [n] granule position of each page's first group
    uint32_t *ws_pair_size;  // [n*hkv] granules per (page, head) K+V pair
    uint64_t *ws_tags;       // [n*hkv] the size pass's findings per (page, head) for the pack pass:
                             // 12-bit: the K group's four tag bytes | the V group's << 32 (null:
                             // not kept); group-adaptive and FP8 tiles: K tile escape bytes |
                             // V tile's << 32
};

// grid of a warp-per-item encoder pass with 8-warp CTAs: one wave of `per_sm` CTAs per
// SM, fewer when there are fewer items than warps
inline unsigned enc_warp_grid(int64_t items, int sms, int per_sm)
{
    const int64_t want = (items + 7) / 8, wave = (int64_t)(sms > 0 ? sms : 1) * per_sm;
    return (unsigned)(want < wave ? (want > 0 ? want : 1) : wave);
}

inline size_t encode_ws_bytes(int n, int hkv)
{
    const size_t a = ((size_t)n * 4 + 15) / 16 * 16;
    return 16 + 2 * a + ((size_t)n * hkv * 4 + 15) / 16 * 16 + (size_t)n * hkv * 8;
}
// byte offset of ws_tags in the encoder workspace
inline size_t encode_ws_tags_offset(int n, int hkv)
{
    const size_t a = ((size_t)n * 4 + 15) / 16 * 16;
    return 16 + 2 * a + ((size_t)n * hkv * 4 + 15) / 16 * 16;
}

struct DecodeParams {
    int hkv;
    int n;
    const uint64_t *meta;
    int64_t num_meta_pages;
    const uint8_t *arena;
    uint64_t arena_bytes;
    const int32_t *page;
    uint16_t *out;
    uint32_t *status;
    const uint32_t *meta32;  // group-adaptive tiles
    const uint8_t *ga_bases;
};

// Attention work split: grid = C CTAs over the flattened (sequence, KV head, page)
// list; partial results live in U + C - 1 slots (U = batch * Hkv units).
constexpr int kCtasPerSm = 3;
constexpr int kMinPagesPerCta = 4;
constexpr int kMaxBatch = 1024;

struct AttnParams {
    int batch, hkv, G, max_pages;
    int grid;  // C
    const uint16_t *q;
    const int32_t *page_ids, *seq_lens, *tail_page;
    const uint64_t *meta;
    const uint32_t *meta32;   // group-adaptive tiles: entries
    const uint8_t *ga_bases;  // group-adaptive tiles: [hkv][2][2][128]
    int64_t num_meta_pages;
    const uint8_t *arena;
    uint64_t arena_bytes;
    int64_t num_raw_pages;
    float *out;
    float *part_o;     // [slots][4 or 8][128] (heads per slot: attn_slot_heads(G))
    float *part_ml;    // [slots][4 or 8][2]
    uint32_t *status;
    float scale_log2;  // log2(e) / sqrt(128)
    // 1: launched as programmatic dependents (KVZ_ATTN_OVERLAP_PREVIOUS); 2: the same, after a
    // kernel that writes nothing this one reads or writes (the prefix kernel)
    int overlap;
};

inline size_t attn_slots(int batch, int hkv, int grid) { return (size_t)batch * hkv + grid - 1; }
// heads per partial slot: 4 for G <= 4, 8 for G = 5..8
inline int attn_slot_heads(int G) { return G > 4 ? 8 : 4; }

// workspace layout: part_o, part_ml
inline size_t attn_ws_bytes(int batch, int hkv, int grid, int G = 4)
{
    size_t slots = attn_slots(batch, hkv, grid);
    const size_t gs = (size_t)attn_slot_heads(G);
    return slots * gs * 128 * 4 + slots * gs * 2 * 4;
}

// New tokens into raw pages (append.cu).  Strides in elements.
struct AppendParams {
    int tokens, hq, hkv, rot, axes;
    bool neighbours;  // pairs (2i, 2i + 1) instead of (i, i + rot / 2)
    float scale;      // on the sines and cosines
    const uint16_t *q, *k, *v;
    int64_t q_token, q_head, k_token, k_head, v_token, v_head;
    const int32_t *slots, *positions;  // [tokens], [axes][tokens]
    const uint64_t *rope;              // [rot / 2][2]: turns per position (2^-64 units), axis
    uint16_t *q_out, *raw_pool;
    int64_t num_raw_pages;
    uint32_t *status;
    int rows_per_block;  // set by the launcher
    bool streaming;      // the same: results written past L2
    // norm weights (null: that operand is not normed), BF16 or (norm_f32) fp32; a head's begin norm_head values
    // behind the one before's
    const void *q_norm, *k_norm;
    int q_norm_head, k_norm_head;
    bool norm_f32;
    float eps;
};
cudaError_t launch_append(AppendParams P, int sms, cudaStream_t stream);

// Step tables from lengths, and pages given back (plan.cu).
struct PlanParams {
    int batch, tokens, num_rows, width, free_capacity;
    const int32_t *rows, *new_tokens, *lens;
    int32_t *tables;  // [num_rows][width]
    const int32_t *free_pages, *free_count;
    int32_t *q_start, *seq_lens, *page_ids, *positions, *slots;
    int32_t *lens_out, *free_out;  // may be lens and free_count
    int32_t *free_out_pages;       // release: free_pages
    bool vector;                   // rows of page_ids begin at multiples of 16 bytes
    uint32_t *status;
};
cudaError_t launch_plan(const PlanParams &P, bool release, cudaStream_t stream);

// Shared-prefix attention (prefix.cu): the prefix half; the own pages go through AttnParams.
constexpr int kPfxMaxGroups = 256;
struct PrefixParams {
    int batch, hkv, G, num_groups, max_pages;
    int max_tokens;  // most prefix tokens the tables can name
    int unit_rows;   // query rows of a CTA's tile: 128 or 256
    int grid;        // CTAs
    int fold;        // blocks of a stream summed in tensor memory at a time
    bool direct;      // no prefix kernel: the own tokens' kernel reads the prefix too
    uint32_t over_G;  // ceil(2^32 / G): the high half of its product with a row is the row's sequence (G > 1)
    const uint16_t *q;
    const int32_t *group_start, *prefix_ids, *prefix_lens, *prefix_tail;
    const uint64_t *meta;
    int64_t num_meta_pages;
    const uint8_t *arena;
    uint64_t arena_bytes;
    const uint16_t *raw_pool;
    int64_t num_raw_pages;
    float *part_o;   // [slots][2][4][16][32][8]: slot = unit + CTA, stream, 32 rows of the tile, 8 columns, row
    float *part_ml;  // [slots][2][128][2]
    void *out;
    bool out_bf16;
    uint32_t *status;
    float scale_log2;
};

// Query rows per tile: two tiles of 128 share a CTA when the average group fills more than one.
inline int pfx_unit_rows(int batch, int G, int groups) { return (int64_t)batch * G > 128LL * groups ? 256 : 128; }
// Most units (group, KV head, tile) of a call.
inline int64_t pfx_max_units(int batch, int hkv, int G, int groups)
{
    return (int64_t)hkv * (groups + (int64_t)batch * G / pfx_unit_rows(batch, G, groups));
}
inline size_t pfx_part_rows(int64_t units, int grid) { return grid > 0 ? (size_t)(units + grid - 1) * 2 * 128 : 0; }

// Own tokens up to this many pages a sequence go through one block per (sequence, KV head), which
// merges the prefix partials too (own.cu); longer ones are split over CTAs (A.grid > 0).
constexpr int kOwnPages = 64;
// Prefix and own pages of a sequence that this kernel can take together, and whether it should (pages
// that the tables can name, blocks = sequences x KV heads).
constexpr int kDirectPages = 128;
bool prefix_direct(int blocks, int pages, int sms);
cudaError_t launch_own(const AttnParams &A, const PrefixParams &P, int format, const void *map, bool after_prefix,
                       int sms, cudaStream_t stream);
// prefix_map: tensor map of the raw pool with one page's 16 K or V rows x 64 columns a box
cudaError_t launch_prefix(const PrefixParams &P, int format, const void *prefix_map, const AttnParams &A,
                          const void *own_map, int sms, cudaStream_t stream);

// Attention of several new tokens a sequence (chunk.cu).
struct ChunkParams {
    int batch, hkv, G, tokens;
    int max_pages, id_page, id_head;  // page_ids: [batch][max_pages], by KV head with id_head = 1, id_page = hkv
    int len_pages;                    // pages of the table that lengths are cut to,
    bool tail;                        // and whether a raw page may stand behind them
    int window, sinks;                // window 0: all keys (sinks 0 then)
    int tile_tokens;                  // new tokens of a tile: 256 / G
    int grid, fold;                   // CTAs; blocks of a stream summed in tensor memory at a time
    uint32_t over_G;                  // ceil(2^32 / G)
    const uint16_t *q;
    const int32_t *q_start, *page_ids, *seq_lens;
    int64_t num_raw_pages;
    float *part_o;   // [2 grid][8][16][32][8]: slot, 32 rows of the tile, 8 columns, row
    float *part_ml;  // [2 grid][256][2]
    int4 *merge;     // [grid] the unit that a CTA began and did not finish: pieces, rows, first token, KV head
    void *out;
    bool out_bf16;
    uint32_t *status;
    float scale_log2;
};
// 12-bit pages: where they are, and the raw pages and their table that the kernel above reads (table null: none).
struct ChunkCoded {
    const int32_t *page_ids, *tail_page;  // [batch][len_pages], [batch]
    const uint64_t *meta;
    int64_t num_meta_pages;
    const uint8_t *arena;
    uint64_t arena_bytes;
    const uint16_t *raw_pool;
    int64_t num_raw_pages;
    int32_t *table;   // [batch][max_pages][hkv] where a page stands among the restored ones
    uint16_t *pages;  // [places][hkv][2][16][128]
    int32_t places;   // pages that the workspace has room for; those behind them are left out and flagged
};
// map: tensor map of the raw pages read, boxes as for launch_prefix
cudaError_t launch_chunk(const ChunkParams &P, const ChunkCoded &X, const void *map, int sms, cudaStream_t stream);

cudaError_t launch_encode(const EncodeParams &P, cudaStream_t stream);
cudaError_t launch_enc_prepare(const EncodeParams &P, cudaStream_t stream);
cudaError_t launch_encode_sizes(const EncodeParams &P, cudaStream_t stream);
cudaError_t launch_enc_scan(const EncodeParams &P, cudaStream_t stream);
cudaError_t launch_ga_encode(const EncodeParams &P, cudaStream_t stream);
cudaError_t launch_ga_decode(const DecodeParams &P, cudaStream_t stream);
cudaError_t launch_wait_selftest(uint64_t limit_ns, uint32_t *status, uint64_t *out, cudaStream_t stream);
cudaError_t launch_late_writer(const void *src, void *dst, uint64_t bytes, uint64_t delay_ns, cudaStream_t stream);
cudaError_t launch_f8_calibrate(int fmt, int hkv, const uint16_t *raw_pool, int64_t num_raw_pages,
                                const int32_t *pages, int n, uint8_t *bases, uint32_t *status, cudaStream_t stream);
cudaError_t launch_f8_encode(int fmt, const EncodeParams &P, cudaStream_t stream);
cudaError_t launch_f8_decode(int fmt, const DecodeParams &P, cudaStream_t stream);
cudaError_t launch_ga_calibrate(int hkv, const uint16_t *raw_pool, int64_t num_raw_pages, const int32_t *pages, int n,
                                uint8_t *bases, uint32_t *status, cudaStream_t stream);
cudaError_t launch_decode(const DecodeParams &P, cudaStream_t stream);
cudaError_t launch_apply_cursor_updates(const int32_t *idx, const uint32_t *pos, const uint32_t *end, int n,
                                        uint32_t *cursors, int num_cursors, cudaStream_t stream);
// tmap: a CUtensorMap (128-byte object) over the raw pool viewed as
// [num_raw_pages*Hkv*32 rows][128 BF16], box 64 x 32, 128-byte swizzle.
// format: 0 plain BF16 pages, 1 12-bit block groups, 2 group-adaptive tiles,
// 3 / 4 FP8 E4M3 / E5M2 tiles (completed pages; the tail stays BF16)
enum AttnFormat : int { kFmtRaw = 0, kFmtZf = 1, kFmtGa = 2, kFmtF8E4 = 3, kFmtF8E5 = 4 };
cudaError_t launch_attention(const AttnParams &P, int format, const void *tmap, cudaStream_t stream);
// the split kernel alone over raw or 12-bit pages: partials in the workspace, no merge and no output;
// third: weights in three BF16 parts instead of two
cudaError_t launch_attention_partials(const AttnParams &P, int format, const void *tmap, bool third, cudaStream_t stream);
// CTAs per SM both attention kernels can hold at this batch size (the smaller of the two)
cudaError_t attn_ctas_per_sm(int batch, int *out);

}  // namespace kvz
