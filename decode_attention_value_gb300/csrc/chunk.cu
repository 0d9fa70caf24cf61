// chunk.cu -- attention of the new tokens of a batch over a paged cache: prompt chunks of any length, drafts of a
// few tokens and single tokens together, each token with the keys up to its own, or with a sliding window
// and the sequence's first tokens.
//
// Mathematics.  Token i of the n new ones of a sequence of L tokens stands at p = L - n + i and sees the keys j <= p,
// with a window W those with j > p - W or j < sinks.  For one KV head the rows (token, query head of the
// group) of a tile are the rows of a matrix Q: S = Q K^T, P = exp2(S c - m) with scores of unseen keys minus
// infinity, O = P V, with the running maximum m and sum l of each row, O / l at the end.
//
// Bound: the tensor cores for chunks, three products of 128 x 128 x 128 a tile of 128 rows and block of keys (S, and O for
// each part of the weights), and the latency of a row's softmax (2039 tokens behind 30710, 32/8 heads: 1050 us,
// 1.0 PFLOP/s, 1.5 as issued, tensor pipe 70 % busy); the bytes of the pages for few rows (64 single tokens with a
// window of 4096: 184 us, 5.9 TB/s).
//
// Split: a unit is (sequence, KV head, tile of up to 256 rows) and has as many blocks of 128 keys as its rows see; the
// units' blocks are one line, cut into equal ranges, a CTA each, so any mix of chunks and single tokens
// keeps all SMs busy for the same time.  A unit that lies in one range is finished there; the others, at most
// two a CTA, leave a maximum, sum and unnormalised output a row, which a second kernel adds in order.  Blocks
// that no row of a tile sees are not on the line, pages that none sees are not read.
#include <cuda.h>

#include <cstring>

#include "chunk.cuh"
#include "prefix.cuh"
#include "tc.cuh"

namespace kvz {

constexpr int kChPages = kChunkBlock / kPage;
constexpr uint32_t kChUnit = kChunkBlock * kDim * 2;  // K or V of a block, BF16
constexpr uint32_t kChHalf = kChUnit / 2;             // its 64-column halves
constexpr uint32_t kChQTile = 128 * kDim * 2;         // 128 query rows
constexpr uint32_t kChQHalf = kChQTile / 2;
constexpr int kChThreads = 512;
constexpr int kChInfo = 8;  // blocks whose bad pages are remembered
constexpr int kChSegs = 8;  // segments handed out ahead
constexpr uint32_t kChColO = 256;  // tensor memory: scores of the streams, overwritten by their weights; outputs

// Warps: 0-7 softmax (two streams of 128 rows), 8 and 10 copy K and V, 9 issues the products, 11 deals out the
// segments, 12-15 fetch queries.  A tile of more than 128 rows gives stream s the rows [128 s, 128 s + 128), and
// both see every block; of a smaller one both have the same rows and alternate blocks, joined at the end.
struct ChSmem {
    static constexpr int ku = 2, vu = 3, units = ku + vu;
    __host__ __device__ static constexpr int slot(int n, int kv) { return kv ? ku + n % vu : n % ku; }
    __host__ __device__ static constexpr uint32_t phase(int n, int kv) { return (kv ? n / vu : n / ku) & 1; }
    static constexpr int q = 0;
    static constexpr int ring = q + 2 * (int)kChQTile;
    static constexpr int full = ring + units * (int)kChUnit;
    static constexpr int empty = full + units * 8;
    static constexpr int qfull = empty + units * 8;  // [2] a tile of queries is there
    static constexpr int qempty = qfull + 16;        // [2] the products have read it
    static constexpr int sfull = qempty + 16;        // [2] scores of a stream are in tensor memory
    static constexpr int pready = sfull + 16;        // [2][3] its weights of half a block are, third parts
    static constexpr int pused = pready + 48;        // [2] those of the first half have been used
    static constexpr int ofull = pused + 16;         // [2] its output of the segment is complete
    static constexpr int pair = ofull + 16;          // [4] warps of both streams that hold the same rows
    static constexpr int gfull = pair + 32;          // [kChSegs] segments
    static constexpr int gempty = gfull + kChSegs * 8;
    static constexpr int drain = gempty + kChSegs * 8;
    static constexpr int info = drain + 8;            // [kChInfo] bad pages of a block, a bit each
    static constexpr int misc = info + kChInfo * 4;   // tensor memory address, abort flag
    static constexpr int seg = (misc + 16 + 15) / 16 * 16;  // [kChSegs][12]
    static constexpr int xml = seg + kChSegs * 48;          // [2][128] {maximum, sum} of a stream's rows
    static constexpr int bytes = xml + 2 * 128 * 8;
};
static_assert(ChSmem::bytes <= 227 * 1024 && ChSmem::seg % 16 == 0 && ChSmem::xml % 16 == 0, "shared memory");

// Consecutive blocks of one unit.
struct ChSeg {
    int blocks, i0, sb, wb;  // i0: the unit's block that is the first; 0 blocks: no more segments
    int hi, lo, p0, rows;
    int q0, flags, b, slot;  // slot: where the rows' partials go
    __device__ __forceinline__ bool both() const { return flags & 1; }     // the streams share the rows
    __device__ __forceinline__ bool whole() const { return flags & 2; }    // the unit is finished here
    __device__ __forceinline__ int kvh() const { return flags >> 8; }
    __device__ __forceinline__ int block(int j) const { return i0 + j < sb ? i0 + j : wb + i0 + j - sb; }
};

// A bounded wait that gives up for the whole CTA.
struct ChWait {
    uint32_t *status;
    volatile uint32_t *abort;
    bool ok;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity)
    {
        if (!ok) return false;
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t it = 1;; ++it) {
            if (mbar_try_wait(bar, parity)) return true;
            if ((it & 255u) == 0 && (*abort || globaltimer_ns() - t0 > kWaitLimitNs)) {
                atomicOr(status, KVZ_STATUS_TIMEOUT);
                *abort = 1;
                return ok = false;
            }
        }
    }
};

// The lowest n of 32 bits (n any number).
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1; }

// Of keys at .. at + 31, those that a token at position p sees.
__device__ __forceinline__ uint32_t seen_bits(const ChunkParams &P, int p, int at)
{
    uint32_t m = low_bits(p - at + 1);
    if (P.window > 0 && p >= P.window) m &= ~low_bits(p - P.window + 1 - at) | low_bits(P.sinks - at);
    return m;
}

// Sums over the threads before this one, and over all.
__device__ __forceinline__ int64_t ch_scan(int64_t v, int64_t &all, int64_t *red)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t own = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += x;
    }
    if (lane == 31) red[warp] = v;
    __syncthreads();
    int64_t before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kChThreads / 32; ++w) {
        const int64_t x = red[w];
        if (w < warp) before += x;
        all += x;
    }
    __syncthreads();
    return v - own + before;
}

template <int kParts>
__global__ void __launch_bounds__(kChThreads, 1) k_chunk(const ChunkParams P, const __grid_constant__ CUtensorMap tmap)
{
    using S = ChSmem;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_addr(smem);
    if (sbase & 1023u) {  // swizzled operands need 1024-byte alignment
        if (threadIdx.x == 0) atomicOr(P.status, KVZ_STATUS_BAD_INDEX);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile uint32_t *info = reinterpret_cast<volatile uint32_t *>(smem + S::info);
    volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(smem + S::misc);
    if (tid == 0) {
        for (int s = 0; s < S::units; ++s) {
            mbar_init(sbase + S::full + 8 * s, 1);
            mbar_init(sbase + S::empty + 8 * s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(sbase + S::qfull + 8 * s, 64);
            mbar_init(sbase + S::qempty + 8 * s, 1);
            mbar_init(sbase + S::sfull + 8 * s, 1);
            for (int i = 0; i < 3; ++i) mbar_init(sbase + S::pready + 24 * s + 8 * i, 128);
            mbar_init(sbase + S::pused + 8 * s, 1);
            mbar_init(sbase + S::ofull + 8 * s, 1);
        }
        for (int s = 0; s < kChSegs; ++s) {
            mbar_init(sbase + S::gfull + 8 * s, 1);
            mbar_init(sbase + S::gempty + 8 * s, 15);  // every warp but the one that deals them out
        }
        for (int s = 0; s < 4; ++s) mbar_init(sbase + S::pair + 8 * s, 64);
        mbar_init(sbase + S::drain, 1);
        misc[1] = 0;
        fence_barrier_init();
    }
    if (warp == 9) tmem_alloc(sbase + S::misc, 512);
    pdl_wait_primary();
    pdl_launch_dependents();

    // ---- the line of blocks: tiles of each sequence, blocks of each tile; in the ring's memory ----
    int *tp = reinterpret_cast<int *>(smem + S::ring);                 // [batch + 1] tiles before a sequence
    int2 *sq = reinterpret_cast<int2 *>(smem + S::ring + 8192);        // [batch] {new tokens, length}
    unsigned long long *wsum = reinterpret_cast<unsigned long long *>(smem + S::ring + 16384);  // [batch] blocks of a KV head
    int64_t *line = reinterpret_cast<int64_t *>(smem + S::ring + 28672);  // [batch + 1] blocks before a sequence
    int64_t *red = reinterpret_cast<int64_t *>(smem + S::ring + 40960);
    const int per = (P.batch + kChThreads - 1) / kChThreads, b0 = min(P.batch, tid * per), b1 = min(P.batch, b0 + per);
    int64_t all = 0;
    int bad_order = 0;
    {
        int tiles = 0;
        bool cut = false;
        for (int b = b0; b < b1; ++b) {
            const int start = P.q_start[b], end = P.q_start[b + 1], len = P.seq_lens[b];
            const bool ok = 0 <= start && start <= end && end <= P.tokens;
            bad_order |= !ok;
            const ChunkSeq s = chunk_seq(P, ok ? start : 0, ok ? end : 0, len);
            cut |= s.len != len;
            sq[b] = make_int2(s.n, s.len);
            wsum[b] = 0;
            tiles += s.tiles;
        }
        bad_order = __syncthreads_or(bad_order);
        if (bad_order) {  // nothing is computed
            tiles = 0;
            if (tid == 0) atomicOr(P.status, KVZ_STATUS_BAD_ORDER);
        } else if (cut) {
            atomicOr(P.status, KVZ_STATUS_BAD_INDEX);
        }
        int64_t before = ch_scan(tiles, all, red);
        for (int b = b0; b < b1; ++b) {
            tp[b] = (int)before;
            if (!bad_order) before += (sq[b].x + P.tile_tokens - 1) / P.tile_tokens;
        }
        if (tid == 0) tp[P.batch] = (int)all;
    }
    __syncthreads();
    {
        const int tiles = (int)all, each = (tiles + kChThreads - 1) / kChThreads;
        int i = tid * each;
        const int end = min(tiles, i + each);
        if (i < end) {
            int lo = 0, top = P.batch - 1;
            while (lo < top) {  // the last sequence that begins at or before tile i
                const int mid = (lo + top + 1) >> 1;
                if (tp[mid] <= i) lo = mid;
                else top = mid - 1;
            }
            unsigned long long sum = 0;
            for (; i < end; ++i) {
                while (tp[lo + 1] <= i) {
                    if (sum) atomicAdd(&wsum[lo], sum);
                    sum = 0;
                    ++lo;
                }
                sum += chunk_tile(P, sq[lo].x, sq[lo].y, i - tp[lo]).blocks;
            }
            atomicAdd(&wsum[lo], sum);
        }
    }
    __syncthreads();
    int64_t W = 0;
    {
        int64_t mine = 0;
        for (int b = b0; b < b1; ++b) mine += (int64_t)wsum[b] * P.hkv;
        int64_t before = ch_scan(mine, W, red);
        for (int b = b0; b < b1; ++b) {
            line[b] = before;
            before += (int64_t)wsum[b] * P.hkv;
        }
        if (tid == 0) line[P.batch] = W;
    }
    __syncthreads();
    // this CTA's range [x, x_end), and the place of x: sequence, KV head, tile, block of it
    const int c = blockIdx.x, C = (int)min((int64_t)gridDim.x, (W + 1) / 2);
    int64_t x = 0, x_end = 0;
    int at_b = 0, at_h = 0, at_k = 0, at_i = 0;
    if (warp == 11 && c < C) {
        x = chunk_first(c, W, C);
        x_end = chunk_first(c + 1, W, C);
        int top = P.batch - 1;
        while (at_b < top) {
            const int mid = (at_b + top + 1) >> 1;
            if (line[mid] <= x) at_b = mid;
            else top = mid - 1;
        }
        int64_t rem = x - line[at_b];
        const int64_t wb = (int64_t)wsum[at_b];
        at_h = (int)(rem / wb);
        int64_t rest = rem - at_h * wb;
        const int tiles = tp[at_b + 1] - tp[at_b];
        for (int k0 = 0;; k0 += 32) {  // 32 tiles at a time
            const int n = k0 + lane < tiles ? chunk_tile(P, sq[at_b].x, sq[at_b].y, k0 + lane).blocks : 0;
            int sum = n;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, sum, off);
                if (lane >= off) sum += y;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, sum > rest);
            if (past || k0 + 32 >= tiles) {
                const int l = past ? __ffs(past) - 1 : 0;
                at_k = k0 + l;
                at_i = (int)(rest - __shfl_sync(0xffffffffu, sum - n, l));
                break;
            }
            rest -= __shfl_sync(0xffffffffu, sum, 31);
        }
    }
    fence_async_shared();  // the ring's memory goes to the copies
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    ChWait wait{P.status, misc + 1, true};
    auto get = [&](int n) -> ChSeg {  // the CTA's n-th segment; one warp
        ChSeg s{};
        const uint32_t bar = sbase + S::gfull + 8 * (n % kChSegs);
        wait(bar, n / kChSegs & 1);
        if (!__all_sync(0xffffffffu, wait.ok)) {
            wait.ok = false;
            return s;
        }
        const int4 *from = reinterpret_cast<const int4 *>(smem + S::seg + 48 * (n % kChSegs));
        const int4 u = from[0], v = from[1], w = from[2];
        __syncwarp();
        if (lane == 0) mbar_arrive(sbase + S::gempty + 8 * (n % kChSegs));
        return ChSeg{u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w, w.x, w.y, w.z, w.w};
    };

    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 11) {
        // =============================== segments ===============================
        int4 merge = make_int4(0, 0, 0, 0);  // a unit that begins here and ends in another CTA
        ChunkSeq sl{0, 0, 0, 0};             // lane: sequence 32 base + lane
        int base = -1;
        auto seq = [&](int b) -> ChunkSeq {
            if (b / 32 != base) {
                base = b / 32;
                const int i = 32 * base + lane;
                if (i < P.batch) sl = chunk_seq(P, P.q_start[i], P.q_start[i + 1], P.seq_lens[i]);
            }
            return ChunkSeq{__shfl_sync(0xffffffffu, sl.q0, b & 31), __shfl_sync(0xffffffffu, sl.n, b & 31),
                            __shfl_sync(0xffffffffu, sl.len, b & 31), __shfl_sync(0xffffffffu, sl.tiles, b & 31)};
        };
        int n = 0;
        bool ok = true;
        for (bool more = true; more && ok; ++n) {
            ChSeg s{};
            more = x < x_end;
            if (more) {
                const ChunkSeq q = seq(at_b);
                const ChunkTile t = chunk_tile(P, q.n, q.len, at_k);
                s.i0 = at_i;
                s.blocks = (int)min(x_end - x, (int64_t)(t.blocks - at_i));
                s.sb = t.sb;
                s.wb = t.wb;
                s.hi = t.hi;
                s.lo = t.lo;
                s.p0 = t.p0;
                s.rows = t.tokens * P.G;
                s.q0 = q.q0 + at_k * P.tile_tokens;
                const bool ends = at_i + s.blocks == t.blocks;
                s.flags = (s.rows <= 128 ? 1 : 0) | (at_i == 0 && ends ? 2 : 0) | at_h << 8;
                s.b = at_b;
                s.slot = 2 * c + (at_i == 0 ? 1 : 0);
                if (at_i == 0 && !ends) {
                    const int64_t last = x + t.blocks - 1;
                    merge = make_int4((int)(last * C / W) - c + 1, s.rows, s.q0, at_h);
                }
                x += s.blocks;
                at_i = 0;
                if (ends && ++at_k == q.tiles) {
                    at_k = 0;
                    if (++at_h == P.hkv) {
                        at_h = 0;
                        do ++at_b;
                        while (x < x_end && seq(at_b).tiles == 0);
                    }
                }
            }
            ok = __all_sync(0xffffffffu, wait(sbase + S::gempty + 8 * (n % kChSegs), (n / kChSegs & 1) ^ 1));
            if (ok && lane == 0) {
                int4 *to = reinterpret_cast<int4 *>(smem + S::seg + 48 * (n % kChSegs));
                to[0] = make_int4(s.blocks, s.i0, s.sb, s.wb);
                to[1] = make_int4(s.hi, s.lo, s.p0, s.rows);
                to[2] = make_int4(s.q0, s.flags, s.b, s.slot);
                mbar_arrive(sbase + S::gfull + 8 * (n % kChSegs));
            }
        }
        if (lane == 0) P.merge[c] = merge;
    } else if (warp == 8 || warp == 10) {
        // =============================== pages ===============================
        // One lane per page, 32 pages (four blocks) at a time; the ids of the next four blocks are fetched
        // while these are copied.  A page's 16 rows are two boxes, one per 64-column half.
        prefetch_tensormap(&tmap);
        const int kv = warp == 8 ? 0 : 1;
        const uint64_t keep = l2_evict_last();
        auto rows_of = [&](const ChSeg &s, int j0) -> int {  // the page's first row in the pool, -1: not seen, -2: bad, -3: left out
            const int j = j0 + (lane >> 3);
            if (j >= s.blocks) return -1;
            const int page = s.block(j) * kChPages + (lane & 7);
            if (!chunk_page_seen(P, s.lo, s.hi, page * kPage)) return -1;
            const int32_t id = ld_keep_s32(P.page_ids + ((int64_t)s.b * P.max_pages + page) * P.id_page + s.kvh() * P.id_head, keep);
            if (id < 0 || id >= P.num_raw_pages) return P.id_head && id == kPageGone ? -3 : -2;
            return (id * P.hkv + s.kvh()) * 32;
        };
        int seg = 0, n = 0, j0 = 0;
        ChSeg s = get(seg++);
        int cur = rows_of(s, 0);
        bool ok = wait.ok;
        while (s.blocks > 0 && ok) {
            ChSeg s2 = s;
            int j2 = j0 + 4;
            if (j2 >= s.blocks) {
                s2 = get(seg++);
                j2 = 0;
            }
            const int nxt = rows_of(s2, j2);
            if (cur == -2) atomicOr(P.status, KVZ_STATUS_BAD_INDEX);
            const uint32_t good = __ballot_sync(0xffffffffu, cur >= 0), bad = __ballot_sync(0xffffffffu, cur <= -2);
            for (int i = 0; i < 4 && j0 + i < s.blocks; ++i, ++n) {
                const uint32_t live = (good >> (8 * i)) & 0xFFu;
                const int row = __shfl_sync(0xffffffffu, cur, 8 * i + ((lane >> 1) & 7));
                const int slot = S::slot(n, kv);
                const uint32_t fullbar = sbase + S::full + 8 * slot;
                ok = __all_sync(0xffffffffu, wait(sbase + S::empty + 8 * slot, S::phase(n, kv) ^ 1));
                if (!ok) break;
                if (lane == 0) {
                    if (kv == 0) info[n % kChInfo] = (bad >> (8 * i)) & 0xFFu;
                    if (live) mbar_arrive_expect_tx(fullbar, __popc(live) * (kPage * kDim * 2));
                    else mbar_arrive(fullbar);
                }
                __syncwarp();
                if (lane < 2 * kChPages && row >= 0) {
                    const uint32_t dst = sbase + S::ring + slot * kChUnit + (lane & 1) * kChHalf + (lane >> 1) * (kPage * 128);
                    tensor_copy_2d_g2s(dst, &tmap, (lane & 1) * 64, row + kv * kPage, fullbar);
                }
            }
            s = s2;
            j0 = j2;
            cur = nxt;
            ok = ok && wait.ok;
        }
        // never leave with copies in flight: every fill is waited for by the products; after a wait that gave
        // up, 1 ms (copies take microseconds)
        if (!ok) {
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 1000000) {}
        }
    } else if (warp >= 12) {
        // =============================== queries ===============================
        // Two warps a tile of 128 rows; sixteen lanes a row of 256 bytes.  A row is (token, query head of the
        // group); a tile is fetched as soon as the last products of the segment before have read its place.
        const int t = (warp - 12) >> 1, half = warp & 1, ch = lane & 15;
        for (int seg = 0, loads = 0;; ++seg) {
            const ChSeg s = get(seg);
            if (s.blocks == 0) break;
            if (t == 1 && s.both()) continue;
            wait(sbase + S::qempty + 8 * t, (loads & 1) ^ 1);
            ++loads;
            if (!__all_sync(0xffffffffu, wait.ok)) break;
#pragma unroll 4
            for (int i = 0; i < 32; ++i) {
                const int row = 4 * i + 2 * half + (lane >> 4), grow = 128 * t + row;
                const uint32_t dst = sbase + S::q + t * kChQTile + (ch >> 3) * kChQHalf + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
                if (grow < s.rows) {
                    const int tok = P.G == 1 ? grow : (int)__umulhi(grow, P.over_G);
                    cp_async_16(dst, P.q + (((int64_t)(s.q0 + tok) * P.hkv + s.kvh()) * P.G + grow - tok * P.G) * kDim + ch * 8);
                } else {
                    *reinterpret_cast<uint4 *>(smem + (dst - sbase)) = make_uint4(0, 0, 0, 0);
                }
            }
            cp_async_wait_all();
            fence_async_shared();
            mbar_arrive(sbase + S::qfull + 8 * t);
        }
    } else if (warp == 9) {
        // ============================ matrix products ============================
        // One warp issues for both streams in turn, which keeps them half a block apart: one stream's softmax
        // runs while the other's products do.
        constexpr uint32_t kQk = mma_desc(128, kChunkBlock, false), kPv = mma_desc(128, kDim, true);
        const uint32_t go = elect_one(), tm = uniform(tmem), sb = uniform(sbase);
        bool ok = true;
        auto wait_all = [&](uint32_t bar, uint32_t parity) {
            if (ok) ok = __all_sync(0xffffffffu, wait(bar, parity));
            tc_fence_after();
        };
        auto slot_of = [&](int n, int kv) { return uniform(S::slot(n, kv)); };
        auto wait_unit = [&](int n, int kv) { wait_all(sbase + S::full + 8 * S::slot(n, kv), S::phase(n, kv)); };
        // scores of stream s over K block n; give_back: the last product that reads the block
        auto qk = [&](uint32_t s, uint32_t qtile, int n, bool give_back, bool last) {
            const uint32_t slot = slot_of(n, 0);
            const uint64_t a = smem_desc(sb + S::q + qtile * kChQTile, 16, 1024);
            const uint64_t b = smem_desc(sb + S::ring + slot * kChUnit, 16, 1024);
#pragma unroll
            for (int k = 0; k < 8; ++k)  // 16 of the 128 dims: 32 bytes within a half's rows
                mma_ss(go, tm + s * 128, a + (((k >> 2) * kChQHalf + (k & 3) * 32) >> 4),
                       b + (((k >> 2) * kChHalf + (k & 3) * 32) >> 4), kQk, k > 0);
            mma_commit(go, sb + S::sfull + 8 * s);
            if (give_back) mma_commit(go, sb + S::empty + 8 * slot);
            if (last) mma_commit(go, sb + S::qempty + 8 * qtile);
        };
        // output of stream s: its weights of 64 tokens times half of the V block in slot
        auto pv = [&](uint32_t s, uint32_t slot, uint32_t half, bool add) {
            const uint64_t b = smem_desc(sb + S::ring + slot * kChUnit + half * 8 * 1024, kChHalf, 1024);
            const uint32_t w = tm + s * 128 + half * 64, o = tm + kChColO + s * 128;
#pragma unroll
            for (int k = 0; k < 4; ++k)  // 16 tokens: two atoms of V rows, eight columns of weights
#pragma unroll
                for (int part = 0; part < 2; ++part)
                    mma_ts(go, o, w + (k >> 1) * 32 + part * 16 + (k & 1) * 8, b + ((k * 2 * 1024) >> 4), kPv,
                           part || k ? true : add);
            if (kParts == 3 && half == 0) mma_commit(go, sb + S::pused + 8 * s);
        };
        auto pv_third = [&](uint32_t s, uint32_t slot) {  // third parts, all 128 tokens
            const uint64_t b = smem_desc(sb + S::ring + slot * kChUnit, kChHalf, 1024);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                mma_ts(go, tm + kChColO + s * 128, tm + s * 128 + k * 8, b + ((k * 2 * 1024) >> 4), kPv, true);
        };
        uint32_t pphase = 0, qphase = 0;  // bit s
        int n0 = 0;
        for (int seg = 0; ok; ++seg) {
            const ChSeg sg = get(seg);
            if (sg.blocks == 0) break;
            const bool both = sg.both();
            const int nb = sg.blocks, step = both ? 2 : 1;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int j = both ? s : 0;
                if (j >= nb || !ok) break;
                if (!both || s == 0) {
                    wait_all(sbase + S::qfull + 8 * s, qphase >> s & 1);
                    qphase ^= 1u << s;
                }
                if (both || s == 0) wait_unit(n0 + j, 0);
                if (ok) qk(s, both ? 0 : s, n0 + j, both || s == 1, j == nb - 1);
            }
            for (int i = 0; i < (both ? (nb + 1) / 2 : nb) && ok; ++i) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {  // the streams in turn
                    const int j = both ? 2 * i + s : i;
                    if (j >= nb || !ok) break;
                    const uint32_t ph = pphase >> s & 1, pbar = sbase + S::pready + 24 * s, slot = slot_of(n0 + j, 1);
                    if (both || s == 0) wait_unit(n0 + j, 1);
                    wait_all(pbar, ph);
                    if (!ok) break;
                    pv(s, slot, 0, i % P.fold != 0);
                    if (j + step < nb && (both || s == 0)) wait_unit(n0 + j + step, 0);
                    wait_all(pbar + 8, ph);
                    if (!ok) break;
                    pv(s, slot, 1, true);
                    if (kParts == 3) {
                        wait_all(pbar + 16, ph);
                        if (!ok) break;
                        pv_third(s, slot);
                    }
                    pphase ^= 1u << s;
                    if (!both && j == nb - 1) mma_commit(go, sb + S::ofull + 8 * s);
                    if (both || s == 1) mma_commit(go, sb + S::empty + 8 * slot);
                    if (j + step < nb) qk(s, both ? 0 : s, n0 + j + step, both || s == 1, j + step == nb - 1);
                }
            }
            if (both && ok) {  // the streams' rows are joined: both wait for all products
                mma_commit(go, sb + S::ofull);
                mma_commit(go, sb + S::ofull + 8);
            }
            n0 += nb;
        }
        if (!ok || !wait.ok) {  // no product in flight when tensor memory is given back
            mma_commit(go, sbase + S::drain);
            mbar_wait(sbase + S::drain, 0, P.status);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // ================================ softmax ================================
        // Thread = query row.  The running maximum moves, and the output is rescaled, only when it grows by more
        // than 2^8: weights up to 2^8 lose nothing in floating point.  Weights are two BF16 parts, off by at most 2^-17
        // of a weight, a 2^-9 part of a BF16 output's own rounding (one part: 2^-8, which made the error of an output
        // 2.1e-3 where its rounding makes 1.6e-3); fp32 outputs take three (all of it).  The sum is of the
        // unrounded weights.  Every P.fold blocks the output is added to the rows' partials in memory and begins
        // anew: the tensor cores' fp32 sums drop the bits below the accumulator's last.
        const int s = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t tS = tmem + s * 128 + lanes, tO = tmem + kChColO + s * 128 + lanes;
        const uint64_t scale = pack2(P.scale_log2, P.scale_log2), minus = pack2(-1.f, -1.f);
        float2 *xml = reinterpret_cast<float2 *>(smem + S::xml);
        uint32_t sphase = 0, mphase = 0;
        auto meet = [&] {  // the two warps of the quad
            mbar_arrive(sbase + S::pair + 8 * quad);
            wait(sbase + S::pair + 8 * quad, mphase);
            mphase ^= 1;
        };
        int n0 = 0;
        for (int seg = 0;; ++seg) {
            const ChSeg sg = get(seg);
            if (sg.blocks == 0) break;
            const bool both = sg.both();
            const int nb = sg.blocks, row0 = both ? 0 : 128 * s, step = both ? 2 : 1;
            const bool active = row0 + quad * 32 < sg.rows;  // a warp without rows only keeps step
            const int rows = min(32, sg.rows - row0 - quad * 32);
            const int grow = row0 + r, tok = P.G == 1 ? grow : (int)__umulhi(grow, P.over_G);
            // positions: of the row, and of the first and last rows of the stream
            const int p = sg.p0 + tok;
            const int pa = sg.p0 + (P.G == 1 ? row0 : (int)__umulhi(row0, P.over_G));
            const int row9 = min(row0 + 127, sg.rows - 1), pz = sg.p0 + (P.G == 1 ? row9 : (int)__umulhi(row9, P.over_G));
            float m = -INFINITY, l = 0.f;
            // The warp's 32 rows of output, complete in tensor memory and relative to maximum ref, added to
            // their partials.  These are laid out [8 columns][row], so that a store of the warp writes whole lines.
            const int64_t slot0 = (int64_t)sg.slot * kChunkRows + 128 * s + quad * 32;
            float fm = 0.f;  // the partials' maximum
            bool folded = false;
            auto fold = [&](float ref) {
                const float f = !folded || fm == -INFINITY ? 0.f : ex2(fm - ref);
#pragma unroll 1
                for (int w = 0; w < 4; ++w) {
                    uint32_t o[32];
                    tmem_ld32(tO + 32 * w, o);
                    tmem_wait_ld(o);
                    if (lane < rows) {
                        float *at = P.part_o + slot0 * kDim + (4 * w * 32 + lane) * 8;
#pragma unroll
                        for (int i = 0; i < 4; ++i, at += 32 * 8) {
                            if (folded)
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    o[8 * i + k] = __float_as_uint(fmaf(at[k], f, __uint_as_float(o[8 * i + k])));
                            st_global_32b(at, o + 8 * i);
                        }
                    }
                    __syncwarp();  // the tensor memory loads want the whole warp, lanes without a row too
                }
                fm = ref;
                folded = true;
            };
            int mine = 0;
            for (int j = both ? s : 0; j < nb; j += step, ++mine) {
                const int n = n0 + j, at = sg.block(j) * kChunkBlock;
                wait(sbase + S::sfull + 8 * s, sphase);
                sphase ^= 1;
                if (!__all_sync(0xffffffffu, wait.ok)) break;
                tc_fence_after();
                // (the products behind these scores were issued after every earlier product of the stream, so its
                // output is complete)
                const bool fresh = mine % P.fold == 0;  // the output begins anew
                if (fresh && mine > 0 && active) fold(m);
                const uint32_t bad = info[n % kChInfo];
                // keys that no row of the tile sees, or of a bad page: rows of V are made zero, so that weight 0
                // times them is 0
                if (bad || at + kChunkBlock > sg.hi || (at < sg.lo && at + kChunkBlock > P.sinks)) {
                    const int slot = S::slot(n, 1), key = at + r;
                    wait(sbase + S::full + 8 * slot, S::phase(n, 1));
                    if (key >= sg.hi || (key < sg.lo && key >= P.sinks) || (bad >> (r >> 4) & 1)) {
                        uint8_t *to = smem + S::ring + slot * kChUnit + r * 128;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            *reinterpret_cast<uint4 *>(to + 16 * i) = make_uint4(0, 0, 0, 0);
                            *reinterpret_cast<uint4 *>(to + kChHalf + 16 * i) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    fence_async_shared();
                    if (!__all_sync(0xffffffffu, wait.ok)) break;
                }
                // scores of keys that some row of the stream does not see: minus infinity
                const bool part = bad || at + kChunkBlock - 1 > pa ||
                                  (P.window > 0 && at <= pz - P.window && at + kChunkBlock > P.sinks);
                if (part && active) {
#pragma unroll 1
                    for (int w = 0; w < 4; ++w) {
                        uint32_t live = seen_bits(P, p, at + 32 * w);
                        live &= ~((bad >> (2 * w) & 1 ? 0xFFFFu : 0u) | (bad >> (2 * w + 1) & 1 ? 0xFFFF0000u : 0u));
                        uint32_t v[32];
                        tmem_ld32(tS + 32 * w, v);
                        tmem_wait_ld(v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = live >> i & 1 ? v[i] : 0xFF800000u;
                        tmem_st32(tS + 32 * w, v);
                    }
                    tmem_wait_st();
                }
                float u = 0.f;
                if (active) {
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[2][32];
                        tmem_ld32(tS + 64 * h, v[0]);
                        tmem_ld32(tS + 64 * h + 32, v[1]);
                        tmem_wait_ld(v[0]);
                        tmem_wait_ld(v[1]);
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            top[i & 2] = max3(top[i & 2], __uint_as_float(v[0][i]), __uint_as_float(v[0][i + 1]));
                            top[(i & 2) + 1] = max3(top[(i & 2) + 1], __uint_as_float(v[1][i]), __uint_as_float(v[1][i + 1]));
                        }
                    }
                    const float bm = fmaxf(max3(top[0], top[1], top[2]), top[3]) * P.scale_log2;
                    const bool grow_m = mine == 0 || bm > m + 8.f;
                    if (mine > 0 && __any_sync(0xffffffffu, grow_m)) {
                        const float f = grow_m ? (m == -INFINITY ? 0.f : ex2(m - bm)) : 1.f;
                        l *= f;
#pragma unroll 1
                        for (int w = 0; w < 4 && !fresh; ++w) {
                            uint32_t o[32];
                            tmem_ld32(tO + 32 * w, o);
                            tmem_wait_ld(o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st32(tO + 32 * w, o);
                        }
                    }
                    if (grow_m) m = bm;
                    u = m == -INFINITY ? 0.f : m;
                }
                const uint64_t shift = pack2(-u, -u);
                uint64_t sum[2] = {0ull, 0ull};
                uint32_t third[kParts == 3 ? 4 : 1][16];
#pragma unroll(kParts == 3 ? 2 : 1)
                for (int half = 0; half < 2; ++half) {
                    if (active) {
                        uint32_t v[2][32];
                        tmem_ld32(tS + 64 * half, v[0]);
                        tmem_ld32(tS + 64 * half + 32, v[1]);
                        tmem_wait_ld(v[0]);
                        tmem_wait_ld(v[1]);
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            uint32_t hi2[16], lo2[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                float p0, p1;
                                unpack2(fma2(pack2(__uint_as_float(v[w][2 * i]), __uint_as_float(v[w][2 * i + 1])), scale,
                                             shift),
                                        p0, p1);
                                p0 = ex2(p0);
                                p1 = ex2(p1);
                                const uint64_t e = pack2(p0, p1);
                                sum[i & 1] = add2(sum[i & 1], e);
                                hi2[i] = pack_bf16x2(p0, p1);
                                auto rest = [&](uint64_t y, uint32_t part) {  // y without its BF16 part, exact
                                    return fma2(pack2(__uint_as_float(part << 16), __uint_as_float(part & 0xFFFF0000u)), minus, y);
                                };
                                float r0, r1;
                                const uint64_t d = rest(e, hi2[i]);
                                unpack2(d, r0, r1);
                                lo2[i] = pack_bf16x2(r0, r1);
                                if (kParts == 3) {
                                    unpack2(rest(d, lo2[i]), r0, r1);
                                    third[(kParts == 3 ? 2 * half : 0) + (kParts == 3 ? w : 0)][i] = pack_bf16x2(r0, r1);
                                }
                            }
                            tmem_st16(tS + 64 * half + 32 * w, hi2);
                            tmem_st16(tS + 64 * half + 32 * w + 16, lo2);
                        }
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    mbar_arrive(sbase + S::pready + 24 * s + 8 * half);
                }
                if (kParts == 3) {  // the third parts, over the first half's when they have been used
                    wait(sbase + S::pused + 8 * s, sphase ^ 1);
                    if (!__all_sync(0xffffffffu, wait.ok)) break;
                    tc_fence_after();
                    if (active) {
#pragma unroll
                        for (int w = 0; w < (kParts == 3 ? 4 : 0); ++w) tmem_st16(tS + 16 * w, third[w]);
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    mbar_arrive(sbase + S::pready + 24 * s + 16);
                }
                if (active) {
                    float s0, s1;
                    unpack2(add2(sum[0], sum[1]), s0, s1);
                    l += s0 + s1;
                }
            }
            n0 += nb;
            // ---- the segment's rows: to the output, or to their partials ----
            // (a maximum of minus infinity says that a partial has no key, which is not so where all scores were NaN)
            const float ml = l != l ? 0.f : m;
            wait(sbase + S::ofull + 8 * s, seg & 1);
            if (!__all_sync(0xffffffffu, wait.ok)) break;
            tc_fence_after();
            auto emit = [&](int w, const float (&o)[32], float k) {  // columns 32 w ..
                const int64_t to = (((int64_t)(sg.q0 + tok) * P.hkv + sg.kvh()) * P.G + grow - tok * P.G) * kDim + 32 * w;
                uint32_t y[32];
                if (P.out_bf16) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) y[i] = pack_bf16x2(o[2 * i] * k, o[2 * i + 1] * k);
                    st_global_32b(static_cast<uint16_t *>(P.out) + to, y);
                    st_global_32b(static_cast<uint16_t *>(P.out) + to + 16, y + 8);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(o[i] * k);
#pragma unroll
                    for (int i = 0; i < 4; ++i) st_global_32b(static_cast<float *>(P.out) + to + 8 * i, y + 8 * i);
                }
            };
            if (!both) {
                if (active && !sg.whole()) {
                    fold(m);
                    if (lane < rows) *reinterpret_cast<float2 *>(P.part_ml + (slot0 + lane) * 2) = make_float2(ml, l);
                    __syncwarp();
                } else if (active) {
                    const float f = !folded || fm == -INFINITY ? 0.f : ex2(fm - m), k = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
                    for (int w = 0; w < 4; ++w) {
                        uint32_t v[32];
                        tmem_ld32(tO + 32 * w, v);
                        tmem_wait_ld(v);
                        if (lane < rows) {
                            float o[32];
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(v[i]);
                            if (folded) {
                                const float *at = P.part_o + slot0 * kDim + (4 * w * 32 + lane) * 8;
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] = fmaf(at[(i >> 3) * 256 + (i & 7)], f, o[i]);
                            }
                            emit(w, o, k);
                        }
                        __syncwarp();
                    }
                }
            } else if (active) {
                // both streams hold the same rows: each thread joins half of its row's columns.  A stream that
                // folded leaves all of its output in memory
                const bool fa = (nb + 1) / 2 > P.fold, fb = nb / 2 > P.fold;
                if (s == 0 ? fa : fb) fold(m);
                xml[128 * s + r] = make_float2(ml, l);
                tc_fence_before();
                meet();
                if (!__all_sync(0xffffffffu, wait.ok)) break;
                tc_fence_after();
                const float2 a = xml[r], b = xml[128 + r];
                const float top = fmaxf(a.x, b.x);
                const float ka = a.x == -INFINITY ? 0.f : ex2(a.x - top), kb = b.x == -INFINITY ? 0.f : ex2(b.x - top);
                const float sum = a.y * ka + b.y * kb, k = sum == 0.f ? 0.f : 1.f / sum;
                float *part = P.part_o + ((int64_t)sg.slot * kChunkRows + quad * 32) * kDim;
#pragma unroll 1
                for (int w = 2 * s; w < 2 * s + 2; ++w) {
                    float o[32];
                    uint32_t v[32];
                    tmem_ld32(tmem + kChColO + lanes + 32 * w, v);
                    tmem_wait_ld(v);
                    float *at = part + (4 * w * 32 + lane) * 8;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float y = fa ? (lane < rows ? at[(i >> 3) * 256 + (i & 7)] : 0.f) : __uint_as_float(v[i]);
                        o[i] = ka > 0.f ? y * ka : 0.f;
                    }
                    __syncwarp();
                    if (nb > 1) {
                        tmem_ld32(tmem + kChColO + 128 + lanes + 32 * w, v);
                        tmem_wait_ld(v);
                        const float *bt = at + 128 * kDim;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float y = fb ? (lane < rows ? bt[(i >> 3) * 256 + (i & 7)] : 0.f) : __uint_as_float(v[i]);
                            if (kb > 0.f) o[i] = fmaf(y, kb, o[i]);
                        }
                        __syncwarp();
                    }
                    if (lane < rows) {
                        if (sg.whole()) {
                            emit(w, o, k);
                        } else {
                            uint32_t y[32];
#pragma unroll
                            for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(o[i]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) st_global_32b(at + 256 * i, y + 8 * i);
                        }
                    }
                    __syncwarp();
                }
                if (s == 0 && lane < rows && !sg.whole())
                    *reinterpret_cast<float2 *>(P.part_ml + ((int64_t)sg.slot * kChunkRows + r) * 2) = make_float2(top, sum);
                __syncwarp();
                tc_fence_before();
                meet();  // (the next segment's first products overwrite both outputs)
                if (!__all_sync(0xffffffffu, wait.ok)) break;
            }
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------------
// merge: block (c, g) adds the partials of rows 32 g .. of the unit that CTA c began and did not finish: its own
// and, in order, those of the CTAs behind it.  A warp a row, 32 partials at a time.
// ---------------------------------------------------------------------------------
constexpr int kChMergeThreads = 256;

__global__ void __launch_bounds__(kChMergeThreads) k_chunk_merge(const ChunkParams P)
{
    const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait_primary();
    const int4 unit = P.merge[c];  // pieces, rows, first token, KV head
    if (unit.x == 0) return;
    for (int r = 32 * blockIdx.y + warp; r < min(unit.y, 32 * (int)blockIdx.y + 32); r += kChMergeThreads / 32) {
        RowSum sum;
        auto row = [&](int i) { return (int64_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * kChunkRows + r; };
        for (int i0 = 0; i0 < unit.x; i0 += 32) {
            float2 e = make_float2(-INFINITY, 0.f);
            if (i0 + lane < unit.x) e = *reinterpret_cast<const float2 *>(P.part_ml + row(i0 + lane) * 2);
            sum.add(e.x, e.y, [&](int k) {
                const int64_t at = row(i0 + k);
                return *reinterpret_cast<const float4 *>(P.part_o + (at & ~31ll) * kDim + ((lane >> 1) * 32 + (at & 31)) * 8 +
                                                         (lane & 1) * 4);
            });
        }
        const int tok = r / P.G;
        const float k = sum.l == 0.f ? 0.f : 1.f / sum.l;
        const int64_t to = (((int64_t)(unit.z + tok) * P.hkv + unit.w) * P.G + r - tok * P.G) * kDim + 4 * lane;
        if (P.out_bf16)
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(P.out) + to) =
                make_uint2(pack_bf16x2(sum.o.x * k, sum.o.y * k), pack_bf16x2(sum.o.z * k, sum.o.w * k));
        else
            *reinterpret_cast<float4 *>(static_cast<float *>(P.out) + to) =
                make_float4(sum.o.x * k, sum.o.y * k, sum.o.z * k, sum.o.w * k);
    }
}

// ---------------------------------------------------------------------------------
// 12-bit pages that any new token sees, and the raw tails behind them, as raw pages of the workspace, one behind
// the other in the sequences' order; the table of places goes by the sequence's pages.  Each block works out where
// the pages of its groups of sequences begin, so the work is of the pages seen and not of the table's width.  A warp a
// (page, KV head); tiles are put together in shared memory by 8 x 8 matrices, then written as whole rows.
// ---------------------------------------------------------------------------------
constexpr int kRestoreWarps = 4, kRestorePitch = 272, kRestoreGroups = kRestoreWarps * 32;

__global__ void __launch_bounds__(kRestoreWarps * 32, 6) k_chunk_restore(const ChunkParams P, const ChunkCoded X)
{
    __shared__ __align__(16) uint8_t buf[kRestoreWarps][2][kPage * kRestorePitch];
    __shared__ int64_t begin[kRestoreGroups + 1], red[kRestoreWarps];  // pages before a group, of a warp's groups
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait_primary();
    auto seen = [&](int b, int &len) -> ChunkPages {  // of sequence b
        const int start = P.q_start[b], end = P.q_start[b + 1];
        if (start < 0 || start >= end || end > P.tokens) return ChunkPages{0, 0, 0};  // (out of order: flagged where nothing is computed)
        len = named_tokens(P.seq_lens[b], P.len_pages, true);
        return chunk_pages(P, end - start, len);
    };
    const int per = (P.batch + kRestoreGroups - 1) / kRestoreGroups;  // sequences of a group
    {
        int64_t n = 0;
        for (int b = tid * per; b < min(P.batch, (tid + 1) * per); ++b) {
            int len;
            n += seen(b, len).count();
        }
        const int64_t own = n;
        __syncwarp();
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, n, off);
            if (lane >= off) n += y;
        }
        if (lane == 31) red[warp] = n;
        __syncthreads();
        n -= own;
        for (int w = 0; w < warp; ++w) n += red[w];
        begin[tid] = n;
        if (tid == kRestoreGroups - 1) begin[kRestoreGroups] = n + own;
        __syncthreads();
    }
    const int64_t items = begin[kRestoreGroups] * P.hkv, step = (int64_t)gridDim.x * kRestoreWarps;
    for (int64_t it = (int64_t)blockIdx.x * kRestoreWarps + warp; it < items; it += step) {
        const int64_t place = it / P.hkv;
        const int kvh = (int)(it - place * P.hkv);
        int lo = 0, top = kRestoreGroups - 1;
        while (lo < top) {  // the last group that begins at or before the place: the one that holds it
            const int mid = (lo + top + 1) >> 1;
            if (begin[mid] <= place) lo = mid;
            else top = mid - 1;
        }
        int b = lo * per, len = 0;
        int64_t k = place - begin[lo];
        ChunkPages g = seen(b, len);
        for (; k >= g.count(); g = seen(++b, len)) k -= g.count();
        const int page = g.page((int)k);
        const int64_t at = ((int64_t)b * P.max_pages + page) * P.hkv + kvh;  // in the table
        uint4 *out = reinterpret_cast<uint4 *>(X.pages) + it * 512;
        uint32_t flag = 0;
        const bool coded = page < len / kPage;
        const int32_t id = coded ? X.page_ids[(int64_t)b * P.len_pages + page] : X.tail_page[b];
        if (place >= X.places) {
            flag = KVZ_STATUS_ARENA_FULL;
        } else if (!coded) {
            if (id < 0 || id >= X.num_raw_pages) {
                flag = id == -1 ? KVZ_STATUS_BAD_TAIL : KVZ_STATUS_BAD_INDEX;
            } else {
                const uint4 *from = reinterpret_cast<const uint4 *>(X.raw_pool) + ((int64_t)id * P.hkv + kvh) * 512;
#pragma unroll
                for (int i = 0; i < 16; ++i) out[32 * i + lane] = from[32 * i + lane];
            }
        } else if (id < 0 || id >= X.num_meta_pages) {
            flag = KVZ_STATUS_BAD_INDEX;
        } else {
            uint64_t words[2];
            words[0] = X.meta[((int64_t)id * P.hkv + kvh) * 2];
            words[1] = X.meta[((int64_t)id * P.hkv + kvh) * 2 + 1];
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const uint32_t off = (uint32_t)words[kv], tags = (uint32_t)(words[kv] >> 32);
                if (!tags_valid(tags) || off == KVZ_OFFSET_INVALID || ((uint64_t)off + group_granules(tags)) * kGranule > X.arena_bytes)
                    flag = KVZ_STATUS_BAD_META;
            }
            __syncwarp();  // the last item's rows have been read
            const int mi = lane >> 3, rr = lane & 7;
#pragma unroll
            for (int kv = 0; kv < 2 && !flag; ++kv) {
                const uint8_t *src = X.arena + (uint64_t)(uint32_t)words[kv] * kGranule;
                const int row = rr + 8 * (kv ? mi >> 1 : mi & 1), c8 = kv ? mi & 1 : mi >> 1;
                const uint32_t to = smem_addr(buf[warp][kv]) + row * kRestorePitch + c8 * 16;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t tag = (uint32_t)(words[kv] >> (32 + 8 * j)) & 0xFFu;
                    uint32_t a0[4], a1[4];
                    if (tag == 0xFFu) {
                        const uint4 u = *reinterpret_cast<const uint4 *>(src + 32 * lane), v = *reinterpret_cast<const uint4 *>(src + 32 * lane + 16);
                        a0[0] = u.x; a0[1] = u.y; a0[2] = u.z; a0[3] = u.w;
                        a1[0] = v.x; a1[1] = v.y; a1[2] = v.z; a1[3] = v.w;
                    } else {
                        const uint4 low = *reinterpret_cast<const uint4 *>(src + 16 * lane);
                        const uint2 code = *reinterpret_cast<const uint2 *>(src + 512 + 8 * lane);
                        restore_fragment(low.x, low.y, code.x, tag * 0x01010101u, a0);
                        restore_fragment(low.z, low.w, code.y, tag * 0x01010101u, a1);
                    }
                    if (kv) {
                        stmatrix_x4_trans(to + 64 * j, a0);
                        stmatrix_x4_trans(to + 64 * j + 32, a1);
                    } else {
                        stmatrix_x4(to + 64 * j, a0);
                        stmatrix_x4(to + 64 * j + 32, a1);
                    }
                    src += tag_granules(tag) * kGranule;
                }
            }
            __syncwarp();
            if (!flag)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int row = 2 * (i & 7) + (lane >> 4);
                    out[32 * i + lane] = *reinterpret_cast<const uint4 *>(buf[warp][i >> 3] + row * kRestorePitch + (lane & 15) * 16);
                }
        }
        if (lane == 0) {
            if (flag) atomicOr(P.status, flag);
            X.table[at] = flag ? kPageGone : (int32_t)place;
        }
    }
}

template <int kParts>
static cudaError_t launch_chunk_impl(const ChunkParams &P, const CUtensorMap &map, const cudaLaunchConfig_t &like)
{
    // per process and device: the whole shared memory (an attribute of the function)
    static unsigned long long done = 0;  // bit per device ordinal < 64
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !(dev < 64 && (__atomic_load_n(&done, __ATOMIC_ACQUIRE) >> dev) & 1ull)) {
        e = cudaFuncSetAttribute(k_chunk<kParts>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e == cudaSuccess && dev < 64) __atomic_fetch_or(&done, 1ull << dev, __ATOMIC_ACQ_REL);
    }
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = like;
    cfg.gridDim = dim3(P.grid);
    cfg.blockDim = dim3(kChThreads);
    cfg.dynamicSmemBytes = ChSmem::bytes;
    return cudaLaunchKernelEx(&cfg, k_chunk<kParts>, P, map);
}

cudaError_t launch_chunk(const ChunkParams &P, const ChunkCoded &X, const void *map, int sms, cudaStream_t stream)
{
    CUtensorMap m;
    memcpy(&m, map, sizeof m);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (X.table) {
        const int64_t want = ((int64_t)X.places * P.hkv + kRestoreWarps - 1) / kRestoreWarps, wave = (int64_t)sms * 6;
        cfg.gridDim = dim3((unsigned)(want < 1 ? 1 : want < wave ? want : wave));
        cfg.blockDim = dim3(kRestoreWarps * 32);
        const cudaError_t e = cudaLaunchKernelEx(&cfg, k_chunk_restore, P, X);
        if (e != cudaSuccess) return e;
    }
    cudaError_t e = P.out_bf16 ? launch_chunk_impl<2>(P, m, cfg) : launch_chunk_impl<3>(P, m, cfg);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(P.grid, kChunkRows / 32);
    cfg.blockDim = dim3(kChMergeThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, k_chunk_merge, P);
}

}  // namespace kvz
