// prefix.cuh -- how the work of shared-prefix attention is laid out, for its kernels: groups, units
// (group, KV head, tile of query rows) of blocks of tokens, dealt to CTAs in equal ranges.
#pragma once

#include "kvz_internal.h"

namespace kvz {

constexpr int kPfxBlock = 128;  // tokens of a block: 8 pages

// Units and blocks of group g (0, 0 when it has no sequence or no prefix).
struct PfxGroup {
    int seq0, seqs, len, blocks, tiles;
};

__device__ __forceinline__ PfxGroup pfx_group(const PrefixParams &P, int g)
{
    PfxGroup r;
    r.seq0 = P.group_start[g];
    r.seqs = P.group_start[g + 1] - r.seq0;
    r.len = min(max(P.prefix_lens[g], 0), P.max_tokens);
    r.blocks = r.len / kPfxBlock + (r.len % kPfxBlock != 0);
    r.tiles = r.blocks > 0 ? (r.seqs * P.G + P.unit_rows - 1) / P.unit_rows : 0;
    return r;
}

// One warp: group starts ordered and in range?
__device__ __forceinline__ bool pfx_groups_ok(const PrefixParams &P, int lane)
{
    bool ok = true;
    for (int g = lane; g < P.num_groups; g += 32) ok &= P.group_start[g] <= P.group_start[g + 1];
    ok &= P.group_start[0] >= 0 && P.group_start[P.num_groups] <= P.batch;
    return __all_sync(0xffffffffu, ok);
}

// First block of CTA c's range of W blocks over C CTAs.
__device__ __forceinline__ int pfx_first(int c, int W, int C) { return (int)(((int64_t)c * W + C - 1) / C); }

// Where the prefix partials of sequence b's rows are: units and blocks before its group, blocks in
// all, the group (-1: none).  One warp, from group starts and lengths alone.
struct PfxPlace {
    int units, blocks, all, group;
};

__device__ __forceinline__ PfxPlace pfx_place(const PrefixParams &P, int b, int lane)
{
    PfxPlace r{0, 0, 0, -1};
    if (P.num_groups == 0 || !pfx_groups_ok(P, lane)) return r;
    for (int g = lane; g < P.num_groups; g += 32) {
        const PfxGroup s = pfx_group(P, g);
        const int n = P.hkv * s.tiles;
        if (s.seq0 + s.seqs <= b) {
            r.units += n;
            r.blocks += n * s.blocks;
        } else if (s.seq0 <= b) {
            r.group = g;
        }
        r.all += n * s.blocks;
    }
    r.units = __reduce_add_sync(0xffffffffu, r.units);
    r.blocks = __reduce_add_sync(0xffffffffu, r.blocks);
    r.all = __reduce_add_sync(0xffffffffu, r.all);
    r.group = __reduce_max_sync(0xffffffffu, r.group);
    return r;
}

// The prefix partials of query head hg (within its KV head) of sequence b: item i is a row of
// part_o and part_ml.
struct PfxItems {
    int n, streams, stream;  // a tile's CTAs leave one or two partials of a row
    int64_t first;           // row of the first CTA's
    __device__ __forceinline__ int64_t row(int i) const
    {
        const int cta = streams == 2 ? i >> 1 : i, s = streams == 2 ? i & 1 : stream;
        return first + (int64_t)(2 * cta + s) * 128;
    }
};

__device__ __forceinline__ PfxItems pfx_items(const PrefixParams &P, const PfxPlace &w, int b, int kvh, int hg)
{
    PfxItems r{0, P.unit_rows == 128 ? 2 : 1, 0, 0};
    if (w.group < 0) return r;
    const PfxGroup s = pfx_group(P, w.group);
    if (s.blocks == 0) return r;
    const int all = (b - s.seq0) * P.G + hg, tile = all / P.unit_rows, row = all - tile * P.unit_rows;
    const int ui = kvh * s.tiles + tile, C = min(P.grid, w.all);
    const int64_t first = w.blocks + (int64_t)ui * s.blocks, last = first + s.blocks - 1;
    const int c0 = (int)(first * C / w.all), c1 = (int)(last * C / w.all);
    r.n = (c1 - c0 + 1) * r.streams;
    r.stream = row >> 7;
    r.first = (int64_t)(w.units + ui + c0) * 2 * 128 + (row & 127);
    return r;
}

// A row's partials merged as they come: running maximum, sum and (four columns a lane) output.
struct RowSum {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    // up to 32 partials (lane k: maximum and sum of the k-th, -inf for one without tokens) whose
    // outputs load(k) brings, eight at a time.  Up to eight are loaded before the maxima are known, of
    // more only those with tokens: a tile's CTA with one block leaves an empty partial beside it.
    template <class Load>
    __device__ __forceinline__ void add(float pm, float pl, int n, const Load &load)
    {
        float4 x[8];
        if (n <= 8)
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = k < n ? load(k) : make_float4(0.f, 0.f, 0.f, 0.f);
        float top = pm;
#pragma unroll
        for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        top = fmaxf(top, m);
        const bool none = pm == -INFINITY;
        const float f = m == -INFINITY ? 0.f : exp2f(m - top), w = none ? 0.f : exp2f(pm - top);
        float sum = none ? 0.f : w * pl;
#pragma unroll
        for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        uint32_t have = __ballot_sync(0xffffffffu, !none);
        l = l * f + sum;
        o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
        m = top;
        auto take = [&](const float4 &v, float wk) {
            o.x += wk * v.x;
            o.y += wk * v.y;
            o.z += wk * v.z;
            o.w += wk * v.w;
        };
        if (n <= 8) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float wk = __shfl_sync(0xffffffffu, w, k);
                if (have >> k & 1) take(x[k], wk);  // (one without tokens was not written)
            }
            return;
        }
        while (have) {
            float wk[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int at = __ffs(have) - 1;  // -1: none left
                wk[k] = __shfl_sync(0xffffffffu, w, at & 31);
                if (at < 0) wk[k] = 0.f;
                x[k] = at < 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : load(at);
                have &= have - 1;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) take(x[k], wk[k]);
        }
    }
    // another warp's
    __device__ __forceinline__ void add(float pm, float pl, const float4 &x)
    {
        const float top = fmaxf(m, pm);
        const float f = m == -INFINITY ? 0.f : exp2f(m - top), w = pm == -INFINITY ? 0.f : exp2f(pm - top);
        l = l * f + (pm == -INFINITY ? 0.f : w * pl);
        o = make_float4(o.x * f + w * x.x, o.y * f + w * x.y, o.z * f + w * x.z, o.w * f + w * x.w);
        m = top;
    }
    // the normalised row (zero without a token) to row `at` of the output
    __device__ __forceinline__ void store(const PrefixParams &P, int64_t at, int lane) const
    {
        const float k = l == 0.f ? 0.f : 1.f / l;
        const int64_t to = at * kDim + 4 * lane;
        if (P.out_bf16)
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(P.out) + to) =
                make_uint2(pack_bf16x2(o.x * k, o.y * k), pack_bf16x2(o.z * k, o.w * k));
        else
            *reinterpret_cast<float4 *>(static_cast<float *>(P.out) + to) =
                make_float4(o.x * k, o.y * k, o.z * k, o.w * k);
    }
};

}  // namespace kvz
