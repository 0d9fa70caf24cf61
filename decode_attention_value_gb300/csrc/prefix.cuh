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

__device__ __forceinline__ PfxGroup pfx_group(const PrefixParams &P, int start, int end, int len)
{
    PfxGroup r;
    r.seq0 = start;
    r.seqs = end - start;
    r.len = min(max(len, 0), P.max_tokens);
    r.blocks = r.len / kPfxBlock + (r.len % kPfxBlock != 0);
    r.tiles = r.blocks > 0 ? (r.seqs * P.G + P.unit_rows - 1) / P.unit_rows : 0;
    return r;
}
__device__ __forceinline__ PfxGroup pfx_group(const PrefixParams &P, int g)
{
    return pfx_group(P, P.group_start[g], P.group_start[g + 1], P.prefix_lens[g]);
}

// CTAs that a unit of `blocks` blocks keeps busy: where the two streams take alternate blocks, one per
// two blocks (they run side by side, and the SMs left over compute the own tokens meanwhile).
__device__ __forceinline__ int pfx_unit_ctas(const PrefixParams &P, int blocks)
{
    return P.unit_rows == 128 ? (blocks + 1) / 2 : blocks;
}

// First block of CTA c's range of W blocks over C CTAs.
__device__ __forceinline__ int pfx_first(int c, int W, int C) { return (int)(((int64_t)c * W + C - 1) / C); }

// Where the prefix partials of sequence b's rows are: units and blocks before its group, blocks and
// CTAs in all, the group (-1: none).  One warp, from group starts and lengths alone.
struct PfxPlace {
    int units, blocks, all, ctas, group;
};

__device__ __forceinline__ PfxPlace pfx_place(const PrefixParams &P, int b, int lane)
{
    PfxPlace r{0, 0, 0, 0, -1};
    if (P.num_groups == 0) return r;
    bool ok = true;  // starts in order and in range
    for (int g = lane; g < P.num_groups; g += 32) {
        const int start = P.group_start[g], end = P.group_start[g + 1];
        const PfxGroup s = pfx_group(P, start, end, P.prefix_lens[g]);
        const int n = P.hkv * s.tiles;
        ok &= 0 <= start && start <= end && end <= P.batch;
        if (s.seq0 + s.seqs <= b) {
            r.units += n;
            r.blocks += n * s.blocks;
        } else if (s.seq0 <= b) {
            r.group = g;
        }
        r.all += n * s.blocks;
        r.ctas += n * pfx_unit_ctas(P, s.blocks);
    }
    if (!__all_sync(0xffffffffu, ok)) return PfxPlace{0, 0, 0, 0, -1};
    r.units = __reduce_add_sync(0xffffffffu, r.units);
    r.blocks = __reduce_add_sync(0xffffffffu, r.blocks);
    r.all = __reduce_add_sync(0xffffffffu, r.all);
    r.ctas = min(P.grid, __reduce_add_sync(0xffffffffu, r.ctas));
    r.group = __reduce_max_sync(0xffffffffu, r.group);
    return r;
}

// The prefix partials of query head hg (within its KV head) of sequence b: item i is row
// first + i * step of part_o and part_ml.
struct PfxItems {
    int n, step;  // (step: a multiple of 32)
    int64_t first;
};

__device__ __forceinline__ PfxItems pfx_items(const PrefixParams &P, const PfxPlace &w, int b, int kvh, int hg)
{
    // a tile's CTAs leave two partials of a row, or one of the row's stream
    const bool both = P.unit_rows == 128;
    PfxItems r{0, both ? 128 : 256, 0};
    if (w.group < 0) return r;
    const PfxGroup s = pfx_group(P, w.group);
    if (s.blocks == 0) return r;
    const int all = (b - s.seq0) * P.G + hg, tile = all / P.unit_rows, row = all - tile * P.unit_rows;
    const int ui = kvh * s.tiles + tile, C = w.ctas;
    const int64_t first = w.blocks + (int64_t)ui * s.blocks, last = first + s.blocks - 1;
    const int c0 = (int)(first * C / w.all), c1 = (int)(last * C / w.all);
    r.n = (c1 - c0 + 1) * (both ? 2 : 1);
    r.first = (int64_t)(w.units + ui + c0) * 2 * 128 + row;
    return r;
}

// 16 bytes from global to shared memory, asynchronously; the thread that asked may read them after
// cp_async_wait_all.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Columns 4 lane .. 4 lane + 3 of a row of part_o, which holds 32 rows as [8 columns][row].
__device__ __forceinline__ const float4 *pfx_part(const PrefixParams &P, int64_t row, int lane)
{
    return reinterpret_cast<const float4 *>(P.part_o + (row & ~31ll) * kDim + ((lane >> 1) * 32 + (row & 31)) * 8 + (lane & 1) * 4);
}

// A row's partials merged as they come: running maximum, sum and (four columns a lane) output.
struct RowSum {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    // Up to 32 partials join (lane k: maximum and sum of the k-th, -inf for one without tokens): the
    // lane's factor of its partial's output, and which have tokens (the others' were not written).
    struct Join {
        float w;
        uint32_t have;
    };
    __device__ __forceinline__ Join join(float pm, float pl)
    {
        float top = pm;
#pragma unroll
        for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        top = fmaxf(top, m);
        const bool none = pm == -INFINITY;
        const float f = m == -INFINITY ? 0.f : exp2f(m - top), w = none ? 0.f : exp2f(pm - top);
        float sum = none ? 0.f : w * pl;
#pragma unroll
        for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        l = l * f + sum;
        o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
        m = top;
        return Join{w, __ballot_sync(0xffffffffu, !none)};
    }
    __device__ __forceinline__ void take(const float4 &v, float w)
    {
        o.x += w * v.x;
        o.y += w * v.y;
        o.z += w * v.z;
        o.w += w * v.w;
    }
    // the same with outputs that load(k) brings, eight at a time
    template <class Load>
    __device__ __forceinline__ void add(float pm, float pl, const Load &load)
    {
        Join j = join(pm, pl);
        while (j.have) {
            float4 x[8];
            float w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int at = __ffs(j.have) - 1;  // -1: none left
                w[k] = __shfl_sync(0xffffffffu, j.w, at & 31);
                if (at < 0) w[k] = 0.f;
                x[k] = at < 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : load(at);
                j.have &= j.have - 1;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) take(x[k], w[k]);
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
