// own.cu -- the own tokens of sequences that share prefixes, when there are few: one block per
// (sequence, KV head) computes their attention and merges the prefix's partials into the output.
//
// The split kernel of attention.cu deals pages out evenly, which long sequences need; for a
// hundred own tokens a sequence its segments are a few pages each, and their partials, written
// and merged by a third kernel, cost more than the pages: 128 sequences x 8 query heads a KV head
// with 0..200 own tokens took 56 us behind the prefix kernel, 52 MB of pages at 8 us.  Here the
// partials never leave the block.
//
// Short prefixes of few sequences come here too (P.direct): every block reads its group's prefix pages
// before its own, from L2 after the first, and there is no other kernel to wait for.
//
// A warp takes every fourth (eighth, sixteenth) page, one or two in flight in its own shared-memory stages, and runs the
// m16n8k16 products of attention.cu on it: S^T = K Q^T with the query heads in the columns, a
// running softmax, O^T += V^T P^T with P as two BF16 parts (three for fp32 outputs).  The block's
// warps leave their states in shared memory; then each head's warp adds the states and the prefix
// partials, in order.
//
// Bound: the latency of a block's dependent reads (lengths and page ids, pages, partials), so those
// of a kind are issued together, and as many warps and blocks as fit run at once (1024 blocks behind 128 x 8 heads and 16384 tokens, 52 MB of
// pages and 25 MB of partials: the whole call 90 to 92 us; with two pages in flight and three blocks an SM
// 100 where this took 95).
#include <cuda.h>

#include <cstring>

#include "frags.cuh"
#include "prefix.cuh"

namespace kvz {

// Warps of a block: 16 where every block has an SM to itself, 8 for up to two blocks an SM, else 4 (six
// blocks an SM with one stage a warp: 80 registers a thread, for which the 12-bit variants spill 40 to 48
// bytes; the raw ones fit).  A warp needs about 0.8 us a page, so a sequence's pages are spread
// over as many as there is room for.
constexpr int kOwnPageBytes = 2 * kPage * kDim * 2;
// Shared memory: the warps' stages, which afterwards hold their states and, behind those, outputs of prefix
// partials; room for more of these where it costs no block; a barrier a stage.
__host__ __device__ constexpr int own_states(int warps) { return warps * 8 * kDim * 4; }
__host__ __device__ constexpr int own_items(int warps, int stages) { return min(32, 16 * stages - 8 + (warps > 4 ? 8 : 0)); }
__host__ __device__ constexpr int own_ring(int warps, int stages) { return warps * stages * kOwnPageBytes; }
__host__ __device__ constexpr int own_bars(int warps, int stages)
{
    return max(own_ring(warps, stages), own_states(warps) + warps * own_items(warps, stages) * kDim * 4);
}
__host__ __device__ constexpr int own_smem(int warps, int stages) { return own_bars(warps, stages) + warps * stages * 8; }
static_assert(kOwnPages + 1 <= 32 * 4 && kDirectPages <= 32 * 4, "a lane resolves one page");

template <int kFmt, bool kG8, bool kThird, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, kWarps == 4 ? 6 : kWarps == 8 ? 2 : 1)
    k_own(const AttnParams A, const PrefixParams P, const int after, const int log_stages,
          const __grid_constant__ CUtensorMap tmap)
{
    constexpr bool kCoded = kFmt != kFmtRaw;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ float2 wml[kWarps][8];  // a warp's (maximum, sum) of each head
    const uint32_t sbase = smem_addr(smem);
    if (sbase & 1023u) {  // the swizzled TMA destinations need 1024-byte alignment
        if (threadIdx.x == 0) atomicOr(A.status, KVZ_STATUS_BAD_INDEX);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int b = blockIdx.x / A.hkv, kvh = blockIdx.x % A.hkv, G = A.G;
    if (after == 2) pdl_wait_primary();  // launched while the kernel before it ends
    // ---- the prefix's pages, if they are read here ----
    int group = -1, plen = 0;
    if (P.direct) {
        bool in_order = true, in_range = true;
        for (int i = lane; i < P.num_groups; i += 32) {
            const int start = P.group_start[i], end = P.group_start[i + 1], len = P.prefix_lens[i];
            in_order &= 0 <= start && start <= end && end <= P.batch;
            in_range &= 0 <= len && len <= P.max_tokens;
            if (start <= b && b < end) {
                group = i;
                plen = min(max(len, 0), P.max_tokens);
            }
        }
        in_order = __all_sync(0xffffffffu, in_order);
        if (blockIdx.x == 0 && warp == 0) {
            if (!in_order && lane == 0) atomicOr(A.status, KVZ_STATUS_BAD_ORDER);
            if (in_order && !in_range) atomicOr(A.status, KVZ_STATUS_BAD_INDEX);
        }
        group = in_order ? __reduce_max_sync(0xffffffffu, group) : -1;
        plen = __reduce_max_sync(0xffffffffu, plen);
        if (group < 0) plen = 0;
    }
    const int np = (plen + kPage - 1) / kPage;
    // lane i holds the place of the warp's i-th page, page warp + kWarps i of the prefix's and then the own ones
    const int page = warp + kWarps * lane, mypage = page - np;
    const int len = A.seq_lens[b], L = named_tokens(len, A.max_pages, kCoded);
    int32_t id = -1;
    if (page < np)
        id = kCoded && page == plen / kPage ? P.prefix_tail[group] : P.prefix_ids[(int64_t)group * P.max_pages + page];
    else if (mypage < A.max_pages)
        id = A.page_ids[(int64_t)b * A.max_pages + mypage];
    const int32_t tail = kCoded ? A.tail_page[b] : 0;
    const int stages = 1 << log_stages;
    const uint32_t ring = sbase + warp * stages * kOwnPageBytes, bar0 = sbase + own_bars(kWarps, stages) + warp * stages * 8;
    if (lane == 0) {  // a warp's barriers are its own
        for (int s = 0; s < stages; ++s) mbar_init(bar0 + 8 * s, 1);
        fence_barrier_init();
    }
    __syncwarp();
    if (L != len && tid == 0) atomicOr(A.status, KVZ_STATUS_BAD_INDEX);
    const int n = np + (L + kPage - 1) / kPage;
    const int mine = (n - warp + kWarps - 1) / kWarps;  // pages warp, warp + kWarps, ...

    float o[8][4];
#pragma unroll
    for (int a = 0; a < 8; ++a) o[a][0] = o[a][1] = o[a][2] = o[a][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    enum : uint32_t { kSkip = 0, kPair = 1, kPlain = 2 };
    uint32_t kind = kSkip, tk = 0, tv = 0;
    const uint8_t *srck = nullptr, *srcv = nullptr;
    int row = 0;
    const int tokens = page < np ? plen - page * kPage : L - mypage * kPage;  // from the page's first on
    if (page < n) {
        uint32_t flag = 0;
        if (kCoded && tokens >= kPage) {
            if (id < 0 || id >= A.num_meta_pages) {
                flag = KVZ_STATUS_BAD_INDEX;
            } else {
                const uint64_t *m = A.meta + ((int64_t)id * A.hkv + kvh) * 2;
                const uint64_t mk = m[0], mv = m[1];
                const uint32_t ofk = (uint32_t)mk, ofv = (uint32_t)mv;
                tk = (uint32_t)(mk >> 32);
                tv = (uint32_t)(mv >> 32);
                if (!tags_valid(tk) || !tags_valid(tv) || ofk == KVZ_OFFSET_INVALID || ofv == KVZ_OFFSET_INVALID ||
                    ((uint64_t)ofk + group_granules(tk)) * kGranule > A.arena_bytes ||
                    ((uint64_t)ofv + group_granules(tv)) * kGranule > A.arena_bytes)
                    flag = KVZ_STATUS_BAD_META;
                else
                    kind = kPair;
                srck = A.arena + (uint64_t)ofk * kGranule;
                srcv = A.arena + (uint64_t)ofv * kGranule;
            }
        } else {
            if (kCoded && page >= np) id = tail;
            if (id < 0 || id >= A.num_raw_pages) {
                flag = kCoded && id == -1 ? KVZ_STATUS_BAD_TAIL : KVZ_STATUS_BAD_INDEX;
            } else {
                kind = kPlain;
                row = (id * A.hkv + kvh) * 32;
            }
        }
        if (flag) atomicOr(A.status, flag);
    }
    auto issue = [&](int i) {  // the warp's i-th page into its stage
        if (lane != i) return;
        const uint32_t bar = bar0 + 8 * (i & (stages - 1)), dst = ring + (i & (stages - 1)) * kOwnPageBytes;
        if (kind == kPair) {
            const uint32_t bk = group_granules(tk) * kGranule, bv = group_granules(tv) * kGranule;
            mbar_arrive_expect_tx(bar, bk + bv);
            bulk_copy_g2s(dst, srck, bk, bar);
            bulk_copy_g2s(dst + bk, srcv, bv, bar);
        } else if (kind == kPlain) {
            mbar_arrive_expect_tx(bar, kOwnPageBytes);
            tensor_copy_2d_g2s(dst, &tmap, 0, row, bar);
            tensor_copy_2d_g2s(dst + 4096, &tmap, 64, row, bar);
        } else {
            mbar_arrive(bar);
        }
    };
    for (int i = 0; i < stages && i < mine; ++i) issue(i);

    // ---- while the pages come: the queries, and where the prefix's partials are ----
    // B operand of QK^T, column = head (n % 4 when G <= 4).  Plain loads: the kernel before this one may
    // have written q, and read-only loads may be moved over the wait for it
    uint32_t qf[8][2];
    const int qhead = kG8 ? g : (g & 3);
    const bool qhas = qhead < G;
    const uint32_t *qg = reinterpret_cast<const uint32_t *>(
        A.q + ((int64_t)b * A.hkv * G + (int64_t)kvh * G + (qhas ? qhead : 0)) * kDim);
#pragma unroll
    for (int kt = 0; kt < 8; ++kt) {
        qf[kt][0] = qhas ? qg[8 * kt + t] : 0u;
        qf[kt][1] = qhas ? qg[8 * kt + t + 4] : 0u;
    }
    const PfxPlace where = after == 1 ? pfx_place(P, b, lane) : PfxPlace{0, 0, 0, 0, -1};

    bool ok = true;
    for (int i = 0; i < mine && ok; ++i) {
        const int s = i & (stages - 1);
        ok = __all_sync(0xffffffffu, mbar_wait(bar0 + 8 * s, (i >> log_stages) & 1, A.status));
        const uint32_t what = __shfl_sync(0xffffffffu, kind, i);
        if (ok && what != kSkip) {
            const uint32_t sta = ring + s * kOwnPageBytes;
            const uint8_t *st = smem + (sta - sbase);
            const uint32_t tagk = __shfl_sync(0xffffffffu, tk, i), tagv = __shfl_sync(0xffffffffu, tv, i);
            const int valid = min(kPage, __shfl_sync(0xffffffffu, tokens, i));
            // ---- S^T = K Q^T over the page's 16 tokens ----
            float sc[4] = {0.f, 0.f, 0.f, 0.f};
            uint32_t off = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t a0[4], a1[4];
                if (kCoded && what == kPair) {
                    const uint32_t tag = (tagk >> (8 * j)) & 0xFFu;
                    block_frags(st + off, tag, lane, a0, a1);
                    off += tag_granules(tag) * kGranule;
                } else {
                    raw_k_frag(sta, j, 0, lane, a0);
                    raw_k_frag(sta, j, 1, lane, a1);
                }
                mma_bf16_16816(sc, a0, qf[2 * j][0], qf[2 * j][1]);
                mma_bf16_16816(sc, a1, qf[2 * j + 1][0], qf[2 * j + 1][1]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[e] *= A.scale_log2;
            if (valid < kPage) {
                if (g >= valid) sc[0] = sc[1] = -INFINITY;
                if (g + 8 >= valid) sc[2] = sc[3] = -INFINITY;
            }
            // ---- running softmax (a column's 16 tokens: lanes with equal t) ----
            float x0 = fmaxf(sc[0], sc[2]), x1 = fmaxf(sc[1], sc[3]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, d));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, d));
            }
            const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
            if (__any_sync(0xffffffffu, n0 > m0 || n1 > m1)) {
                const float f0 = n0 == -INFINITY ? 1.f : exp2f(m0 - n0), f1 = n1 == -INFINITY ? 1.f : exp2f(m1 - n1);
#pragma unroll
                for (int a = 0; a < 8; ++a) {
                    o[a][0] *= f0;
                    o[a][2] *= f0;
                    o[a][1] *= f1;
                    o[a][3] *= f1;
                }
                l0 *= f0;
                l1 *= f1;
                m0 = n0;
                m1 = n1;
            }
            const float u0 = m0 == -INFINITY ? 0.f : m0, u1 = m1 == -INFINITY ? 0.f : m1;
            const float p0 = exp2f(sc[0] - u0), p1 = exp2f(sc[1] - u1), p2 = exp2f(sc[2] - u0), p3 = exp2f(sc[3] - u1);
            l0 += p0 + p2;
            l1 += p1 + p3;
            // P as high and low BF16 parts: for G <= 4 in columns h and h + 4 of one product, else
            // in two products; a product for the third part (columns h)
            const float r0 = p0 - bf16_round(p0), r1 = p1 - bf16_round(p1);
            const float r2 = p2 - bf16_round(p2), r3 = p3 - bf16_round(p3);
            const bool low = !kG8 && t >= 2;
            const uint32_t pb0 = movmatrix_trans(low ? pack_bf16x2(r0, r1) : pack_bf16x2(p0, p1));
            const uint32_t pb1 = movmatrix_trans(low ? pack_bf16x2(r2, r3) : pack_bf16x2(p2, p3));
            uint32_t pl0 = 0, pl1 = 0;
            if (kG8) {
                pl0 = movmatrix_trans(pack_bf16x2(r0, r1));
                pl1 = movmatrix_trans(pack_bf16x2(r2, r3));
            }
            uint32_t pt0 = 0, pt1 = 0;
            if (kThird) {
                pt0 = movmatrix_trans(low ? 0u : pack_bf16x2(r0 - bf16_round(r0), r1 - bf16_round(r1)));
                pt1 = movmatrix_trans(low ? 0u : pack_bf16x2(r2 - bf16_round(r2), r3 - bf16_round(r3)));
            }
            // ---- O^T += V^T P^T ----
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t a[2][4];
                if (kCoded && what == kPair) {
                    const uint32_t tag = (tagv >> (8 * j)) & 0xFFu;
                    block_frags(st + off, tag, lane, a[0], a[1]);  // V right after K
                    off += tag_granules(tag) * kGranule;
                } else {
                    raw_v_frag(sta, j, 0, lane, a[0]);
                    raw_v_frag(sta, j, 1, lane, a[1]);
                    if (valid < kPage) {
                        mask_v_frag(a[0], lane, valid);
                        mask_v_frag(a[1], lane, valid);
                    }
                }
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    mma_bf16_16816(o[2 * j + f], a[f], pb0, pb1);
                    if (kG8) mma_bf16_16816(o[2 * j + f], a[f], pl0, pl1);
                    if (kThird) mma_bf16_16816(o[2 * j + f], a[f], pt0, pt1);
                }
            }
        }
        __syncwarp();
        if (ok && i + stages < mine) issue(i + stages);
    }
    // (after a wait that gave up, the copy it waited for may land late: microseconds)
    if (!ok) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000) {}
    }

    // ---- the warp's state to shared memory ----
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, d);
        l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    if (!kG8) {  // columns h and h + 4: the high and low parts of P
#pragma unroll
        for (int a = 0; a < 8; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[a][e] += __shfl_xor_sync(0xffffffffu, o[a][e], 2);
    }
    __syncthreads();  // every page has been read: the ring holds the states now
    float *states = reinterpret_cast<float *>(smem);  // [warp][8 heads][128]
    if (kG8 || t < 2) {
        const int h0 = 2 * t, h1 = 2 * t + 1;
        if (g == 0) {
            wml[warp][h0] = make_float2(m0, l0);
            wml[warp][h1] = make_float2(m1, l1);
        }
#pragma unroll
        for (int a = 0; a < 8; ++a) {
            float *to = states + (warp * 8 + h0) * kDim + 16 * a + g;
            to[0] = o[a][0];
            to[kDim] = o[a][1];
            to[8] = o[a][2];
            to[kDim + 8] = o[a][3];
        }
    }
    __syncthreads();

    // ---- a head at a time: the states, then the prefix's partials ----
    const int heads = G <= 1 ? 1 : G <= 2 ? 2 : G <= 4 ? 4 : 8;
    const int share = kWarps > heads ? kWarps / heads : 1;  // warps of a head
    const int part = warp % share;
    const int most_items = own_items(kWarps, stages);  // 8 to 24
    const uint32_t items = sbase + own_states(kWarps) + warp * most_items * kDim * 4 + lane * 16;
    PfxItems pre = pfx_items(P, where, b, kvh, min(warp / share, G - 1));
    if (after == 1) pdl_wait_primary();  // the prefix partials are complete
    for (int h0 = 0; h0 < G; h0 += kWarps / share) {  // (uniform: the barrier below)
        const int h = h0 + warp / share;
        RowSum sum;
        if (h < G) {
            for (int w = part; w < kWarps; w += share)
                    sum.add(wml[w][h].x, wml[w][h].y, *reinterpret_cast<const float4 *>(states + (w * 8 + h) * kDim + 4 * lane));
            if (h0 > 0) pre = pfx_items(P, where, b, kvh, h);
            // the prefix's: as many at once as the warp's part of the ring holds, copied while their maxima come
            const int64_t step = (int64_t)share * pre.step;
            int64_t row = pre.first + (int64_t)part * pre.step;
            for (int left = (pre.n - part + share - 1) / share; left > 0; left -= most_items, row += most_items * step) {
                const int count = min(most_items, left);
                const float4 *from = pfx_part(P, row, lane);
#pragma unroll 4
                for (int k = 0; k < count; ++k, from += step * (kDim / 4)) cp_async_16(items + k * (kDim * 4), from);
                float2 e = make_float2(-INFINITY, 0.f);
                if (lane < count) e = *reinterpret_cast<const float2 *>(P.part_ml + (row + lane * step) * 2);
                const RowSum::Join j = sum.join(e.x, e.y);
                cp_async_wait_all();
                const float4 *at = reinterpret_cast<const float4 *>(smem + (items - sbase));
#pragma unroll 4
                for (int k = 0; k < count; ++k) {
                    float4 v = at[k * (kDim / 4)];
                    if (!(j.have >> k & 1)) v = make_float4(0.f, 0.f, 0.f, 0.f);  // (was not written)
                    sum.take(v, __shfl_sync(0xffffffffu, j.w, k));
                }
            }
        }
        if (share > 1) {  // (one turn of the loop, since kWarps / share = heads >= G: all warps meet here)
            __syncthreads();
            if (part > 0 && h < G) {
                *reinterpret_cast<float4 *>(states + warp * 8 * kDim + 4 * lane) = sum.o;
                if (lane == 0) wml[warp][0] = make_float2(sum.m, sum.l);
            }
            __syncthreads();
            if (part > 0) continue;
            for (int w = warp + 1; w < warp + share; ++w)
                sum.add(wml[w][0].x, wml[w][0].y, *reinterpret_cast<const float4 *>(states + w * 8 * kDim + 4 * lane));
        }
        if (h < G) sum.store(P, (int64_t)blockIdx.x * G + h, lane);
    }
}

// Measured, us, here against the prefix kernel and this one behind it (4 query heads a KV head, 40 own
// tokens): up to a block an SM, 16 warps, raw pages of 256 / 1024 / 1900 tokens 6.7 / 9.7 / 12.5 against
// 10.5 / 10.8 / 11.4, 12-bit pages 8.8 / 14.3 / 20 against 15.9 / 15.7 / 16.7; 256 blocks of eight warps,
// raw, 512 / 1024 tokens 10.2 / 14.2 against 12.0 / 12.7, 12-bit 14.6 / 22 against 17 / 17.7; 512 blocks, 128 /
// 256 tokens 8.2 / 10.6 against 12.2 / 12.7, 12-bit 12 / 18 against 17 / 17.5; 1024 blocks, 128 / 256
// tokens 13.8 / 18.5 against 17.5 / 17.9, 12-bit 22 / 31 against 24 / 25.
bool prefix_direct(int blocks, int pages, int sms)
{
    return pages <= (blocks <= sms ? 80 : blocks <= 2 * sms ? 46 : blocks <= 4 * sms ? 20 : 12);
}

template <int kFmt, bool kG8, bool kThird, int kWarps>
static cudaError_t launch_own_impl(const AttnParams &A, const PrefixParams &P, const CUtensorMap &map, bool after, int sms,
                                   cudaStream_t stream)
{
    // per process and device: more shared memory than the default (an attribute of the function)
    static unsigned long long done = 0;  // bit per device ordinal < 64
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !(dev < 64 && (__atomic_load_n(&done, __ATOMIC_ACQUIRE) >> dev) & 1ull)) {
        e = cudaFuncSetAttribute(k_own<kFmt, kG8, kThird, kWarps>, cudaFuncAttributeMaxDynamicSharedMemorySize, own_smem(kWarps, kWarps == 4 ? 2 : 1));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(k_own<kFmt, kG8, kThird, kWarps>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        if (e == cudaSuccess && dev < 64) __atomic_fetch_or(&done, 1ull << dev, __ATOMIC_ACQ_REL);
    }
    if (e != cudaSuccess) return e;
    // pages in flight: two a warp for up to three blocks of four warps an SM, else one
    const int blocks = A.batch * A.hkv, log_stages = kWarps == 4 && blocks <= 3 * sms ? 1 : 0;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = own_smem(kWarps, 1 << log_stages);
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_own<kFmt, kG8, kThird, kWarps>, A, P, after ? 1 : 2, log_stages, map);
}

template <int kFmt, bool kG8>
static cudaError_t launch_own_of(const AttnParams &A, const PrefixParams &P, const CUtensorMap &map, bool after, int sms,
                                 cudaStream_t stream)
{
    const int blocks = A.batch * A.hkv;
    if (blocks <= sms)
        return P.out_bf16 ? launch_own_impl<kFmt, kG8, false, 16>(A, P, map, after, sms, stream)
                          : launch_own_impl<kFmt, kG8, true, 16>(A, P, map, after, sms, stream);
    if (blocks <= 2 * sms)
        return P.out_bf16 ? launch_own_impl<kFmt, kG8, false, 8>(A, P, map, after, sms, stream)
                          : launch_own_impl<kFmt, kG8, true, 8>(A, P, map, after, sms, stream);
    return P.out_bf16 ? launch_own_impl<kFmt, kG8, false, 4>(A, P, map, after, sms, stream)
                      : launch_own_impl<kFmt, kG8, true, 4>(A, P, map, after, sms, stream);
}

cudaError_t launch_own(const AttnParams &A, const PrefixParams &P, int format, const void *map, bool after_prefix, int sms,
                       cudaStream_t stream)
{
    CUtensorMap m;
    memcpy(&m, map, sizeof m);
    if (format == kFmtRaw)
        return A.G > 4 ? launch_own_of<kFmtRaw, true>(A, P, m, after_prefix, sms, stream)
                       : launch_own_of<kFmtRaw, false>(A, P, m, after_prefix, sms, stream);
    return A.G > 4 ? launch_own_of<kFmtZf, true>(A, P, m, after_prefix, sms, stream)
                   : launch_own_of<kFmtZf, false>(A, P, m, after_prefix, sms, stream);
}

}  // namespace kvz
