// plan.cu -- the tables of a serving step, built on the GPU from the requests' lengths: pages for the new
// tokens out of a free list, the requests' block tables, and each new token's position and slot.
//
// Mathematics.  Request b has lens[row] = l tokens and gets n more.  With c(x) = ceil(x / 16) it holds c(l) pages and
// takes c(l + n) - c(l); sums over the requests before it say where its tokens begin in the batch and which pages
// of the free list are its own, so every value is a function of two prefix sums and nothing is taken by atomics: the
// same lengths give the same tables.
//
// Bound: launch and a chain of dependent reads (rows, lengths, prefix sums, pages): 256 requests x 512 pages
// 10.3 us, 61 prompts of 29 K tokens x 2048 pages 13.1 us.
//
// Split: one cluster of eight blocks.  Each works out both sums itself (a thread a request, 4 KB of
// lengths), they meet once, so that everything that a call may update in place has been read, and then
// share the table's rows and the tokens.  (A second kernel for the updates in place is a launch more.)
#include "kvz_device.cuh"
#include "kvz_internal.h"

namespace kvz {

constexpr int kPlanThreads = kMaxBatch, kPlanCtas = 8;
constexpr int kPlanSeen = 4096;  // places of the rows already named: a quarter full at most

__device__ __forceinline__ void cluster_meet()  // thread by thread: lanes of a warp may come here apart
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Sums of two values over the threads before this one, and over all.
__device__ __forceinline__ void block_sums(int64_t (&v)[2], int64_t (&all)[2], int64_t (*red)[2])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t own[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        own[k] = v[k];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, v[k], off);
            if (lane >= off) v[k] += x;
        }
        if (lane == 31) red[warp][k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        int64_t before = 0, sum = 0;
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            const int64_t x = red[w][k];
            if (w < warp) before += x;
            sum += x;
        }
        v[k] += before - own[k];
        all[k] = sum;
    }
}

// Whether `row` was named by another thread (no more than kMaxBatch rows are).
__device__ __forceinline__ bool named_before(int32_t *seen, int32_t row)
{
    uint32_t at = ((uint32_t)row * 2654435761u) >> 20;
    for (int i = 0; i < kPlanSeen; ++i) {
        const int32_t was = atomicCAS(&seen[at], -1, row);
        if (was == -1) return false;
        if (was == row) return true;
        at = (at + 1) & (kPlanSeen - 1);
    }
    return true;
}

__device__ __forceinline__ int pages_of(int tokens) { return (tokens + kPage - 1) / kPage; }

// Whether id is a page whose rows slots can name.
__device__ __forceinline__ bool page_named(int32_t id) { return id >= 0 && id <= INT32_MAX / kPage; }

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1) k_plan(const PlanParams P)
{
    __shared__ int32_t seen[kPlanSeen];
    __shared__ int64_t red[kPlanThreads / 32][2];
    __shared__ int32_t start[kMaxBatch + 1], have[kMaxBatch], row_of[kMaxBatch], fresh[kMaxBatch], after[kMaxBatch];
    __shared__ uint32_t bad;
    const int tid = threadIdx.x, cta = blockIdx.x, lane = tid & 31;
    const int at = cta * kPlanThreads + tid, step = kPlanCtas * kPlanThreads;  // (counts near 2^31: steps in 32 unsigned bits)
    for (int i = tid; i < kPlanSeen; i += kPlanThreads) seen[i] = -1;
    if (tid == 0) bad = 0;
    pdl_wait_primary();
    __syncthreads();
    // ---- what the requests ask for ----
    const int32_t spare = P.free_count[0];
    int row = -1, len = 0, fresh_tokens = 0, last = 0;  // last: the page that takes its first new tokens
    uint32_t flag = spare < 0 || spare > P.free_capacity ? KVZ_STATUS_BAD_INDEX : 0;
    if (tid < P.batch) {
        row = P.rows[tid];
        if (row >= 0 && row < P.num_rows) {
            len = P.lens[row];
            fresh_tokens = P.new_tokens[tid];
            if (len < 0 || fresh_tokens < 0 || (int64_t)len + fresh_tokens > (int64_t)P.width * kPage)
                flag |= KVZ_STATUS_BAD_INDEX;
            else if (named_before(seen, row))
                flag |= KVZ_STATUS_BAD_ORDER;
            else if (fresh_tokens > 0 && len % kPage != 0)
                last = P.tables[(int64_t)row * P.width + len / kPage];
        } else if (row != -1) {
            flag |= KVZ_STATUS_BAD_INDEX;
        }
    }
    if (flag) {
        atomicOr(&bad, flag);
        len = fresh_tokens = 0;
    }
    int64_t v[2] = {fresh_tokens, pages_of(len + fresh_tokens) - pages_of(len)}, all[2];
    block_sums(v, all, red);
    if (tid == 0 && !bad) {
        if (all[0] > P.tokens) bad = KVZ_STATUS_BAD_INDEX;
        else if (all[1] > spare) bad = KVZ_STATUS_ARENA_FULL;
    }
    __syncthreads();
    // every page that takes a new token is one whose rows slots can name
    const bool fits = bad == 0;
    bool named = page_named(last);
    if (fits)
        for (uint32_t i = tid; i < (uint32_t)all[1]; i += kPlanThreads) named &= page_named(P.free_pages[spare - 1 - (int)i]);
    const uint32_t wrong = __syncthreads_or(!named) ? KVZ_STATUS_BAD_INDEX : 0;
    const bool ok = fits && !wrong;  // else: a step without requests, and nothing changes
    if (tid < P.batch) {
        start[tid] = ok ? (int32_t)v[0] : 0;
        have[tid] = ok && row >= 0 ? pages_of(len) : 0;
        after[tid] = ok && row >= 0 ? len + fresh_tokens : 0;
        row_of[tid] = row;
        fresh[tid] = ok ? spare - 1 - (int32_t)v[1] : 0;  // its first page of the free list, the next ones before it
    }
    if (tid == 0) start[P.batch] = ok ? (int32_t)all[0] : 0;
    if (cta == 0 && tid == 0 && !ok) atomicOr(P.status, fits ? wrong : bad);
    if (P.lens_out != P.lens)
        for (uint32_t i = at; i < (uint32_t)P.num_rows; i += step) P.lens_out[i] = P.lens[i];
    cluster_meet();  // lengths and the free list's count have been read, copied lengths written
    if (cta == 0 && tid < P.batch && ok && row >= 0) P.lens_out[row] = len + fresh_tokens;
    if (cta == 0 && tid == 0) P.free_out[0] = ok ? spare - (int32_t)all[1] : spare;
    if (cta == 1) {
        for (int i = tid; i <= P.batch; i += kPlanThreads) P.q_start[i] = start[i];
        if (tid < P.batch) P.seq_lens[tid] = after[tid];
    }
    // ---- the requests' pages: held ones from their row, the rest from the free list ----
    auto page = [&](int b, int c) -> int32_t {
        return c < have[b] ? P.tables[(int64_t)row_of[b] * P.width + c] : P.free_pages[fresh[b] - (c - have[b])];
    };
    const int segs = (P.width + 127) / 128;
    const int64_t pieces = (int64_t)P.batch * segs;
    for (int64_t s = at >> 5; s < pieces; s += step >> 5) {
        const int b = (int)(s / segs), c0 = (int)(s - (int64_t)b * segs) * 128;
        const int want = pages_of(after[b]);
        int32_t x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = c0 + 4 * lane + k;
            x[k] = c < want ? page(b, c) : -1;
            if (c < want && c >= have[b]) P.tables[(int64_t)row_of[b] * P.width + c] = x[k];
        }
        int32_t *to = P.page_ids + (int64_t)b * P.width + c0 + 4 * lane;
        if (P.vector && c0 + 4 * lane < P.width) {
            *reinterpret_cast<int4 *>(to) = make_int4(x[0], x[1], x[2], x[3]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c0 + 4 * lane + k < P.width) to[k] = x[k];
        }
    }
    // ---- the tokens ----
    for (uint32_t u = at; u < (uint32_t)P.tokens; u += step) {
        const int i = (int)u;
        int32_t pos = 0, slot = -1;
        if (i < start[P.batch]) {
            int lo = 0, hi = P.batch - 1;
            while (lo < hi) {  // the last request that begins at or before i: the one that holds it
                const int mid = (lo + hi + 1) >> 1;
                if (start[mid] <= i) lo = mid;
                else hi = mid - 1;
            }
            pos = after[lo] - (start[lo + 1] - start[lo]) + (i - start[lo]);
            slot = page(lo, pos / kPage) * kPage + pos % kPage;
        }
        P.positions[i] = pos;
        P.slots[i] = slot;
    }
}

// Pages of finished requests back to the end of the free list, the last page of each first, so that the next
// request takes them in the order they were in.  An entry that names no page (given back before from behind a
// window) is passed over, so a row's pages are counted first.  One block: 4 KB of lengths and, twice, the rows' pages.
__global__ void __launch_bounds__(kPlanThreads, 1) k_release(const PlanParams P)
{
    __shared__ int32_t seen[kPlanSeen];
    __shared__ int64_t red[kPlanThreads / 32][2];
    __shared__ int32_t begin[kMaxBatch], held[kMaxBatch], span[kMaxBatch], row_of[kMaxBatch];
    __shared__ uint32_t bad;
    const int tid = threadIdx.x, lane = tid & 31;
    for (int i = tid; i < kPlanSeen; i += kPlanThreads) seen[i] = -1;
    if (tid == 0) bad = 0;
    pdl_wait_primary();
    __syncthreads();
    const int32_t spare = P.free_count[0];
    int row = -1, len = 0;
    uint32_t flag = spare < 0 || spare > P.free_capacity ? KVZ_STATUS_BAD_INDEX : 0;
    if (tid < P.batch) {
        row = P.rows[tid];
        if (row >= 0 && row < P.num_rows) {
            len = P.lens[row];
            if (len < 0 || len > (int64_t)P.width * kPage) flag |= KVZ_STATUS_BAD_INDEX;
            else if (named_before(seen, row)) flag |= KVZ_STATUS_BAD_ORDER;
        } else if (row != -1) {
            flag |= KVZ_STATUS_BAD_INDEX;
        }
    }
    if (flag) atomicOr(&bad, flag);
    span[tid] = flag || row < 0 ? 0 : pages_of(len);
    row_of[tid] = row;
    held[tid] = 0;
    __syncthreads();
    const bool any = bad == 0;
    // a row's pages in order, one warp: f(place in the row, page, how many stand before it); returns how many they are
    auto pages = [&](int b, auto &&f) {
        const int32_t *from = P.tables + (int64_t)row_of[b] * P.width;
        int n = 0;
        for (int c0 = 0; c0 < span[b]; c0 += 256) {  // eight loads at once
            int32_t id[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) id[k] = c0 + 32 * k + lane < span[b] ? from[c0 + 32 * k + lane] : -1;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t live = __ballot_sync(0xffffffffu, page_named(id[k]));
                f(c0 + 32 * k + lane, id[k], n + __popc(live & ((1u << lane) - 1)));
                n += __popc(live);
            }
        }
        return n;
    };
    for (int b = tid >> 5; b < P.batch && any; b += kPlanThreads / 32) {
        const int n = pages(b, [](int, int32_t, int) {});
        if (lane == 0) held[b] = n;
    }
    __syncthreads();
    int64_t v[2] = {held[tid], 0}, all[2];
    block_sums(v, all, red);
    if (tid == 0 && any && all[0] > P.free_capacity - spare) bad = KVZ_STATUS_BAD_INDEX;  // more than there are
    begin[tid] = spare + (int32_t)v[0];
    __syncthreads();
    if (bad) {  // nothing changes
        if (tid == 0) atomicOr(P.status, bad);
        return;
    }
    if (tid < P.batch && row >= 0) P.lens_out[row] = 0;
    if (tid == 0) P.free_out[0] = spare + (int32_t)all[0];
    for (int b = tid >> 5; b < P.batch; b += kPlanThreads / 32)
        pages(b, [&](int c, int32_t id, int nth) {
            if (page_named(id)) P.free_out_pages[begin[b] + held[b] - 1 - nth] = id;
            if (c < span[b]) P.tables[(int64_t)row_of[b] * P.width + c] = -1;
        });
}

cudaError_t launch_plan(const PlanParams &P, bool release, cudaStream_t stream)
{
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(release ? 1 : kPlanCtas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return release ? cudaLaunchKernelEx(&cfg, k_release, P) : cudaLaunchKernelEx(&cfg, k_plan, P);
}

}  // namespace kvz
