// prefix.cu -- decode attention of sequences that share a prefix: the prefix's pages are
// read once for all sequences of a group.
//
// Mathematics.  For one KV head the queries of a group, n sequences x G heads, are the rows
// of one matrix Q.  Over the group's prefix, S = Q K^T and O = exp2(S c - m) V are matrix
// products with many rows, so they run on the tcgen05 tensor cores instead of once per
// sequence: the bytes of the prefix are read n times less often, and the arithmetic per byte
// grows with n G.  The kernel leaves partial results (running maximum m, sum l, unnormalised
// O), which are added in a fixed order: sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i, for up
// to 1024 own tokens a sequence by the kernel that computes those (own.cu), else, with the
// partials of attention.cu's split kernel over the own pages, by the merge below.
//
// Bound: with many rows the tensor cores (256 rows a CTA: 85 clocks a product that takes 64, 56% of
// the pipe's time over the launch; 128 x 8 heads behind 16384 tokens: 71 us of 91); with few rows the
// bytes of the prefix for raw pages (131072 tokens x 32 sequences: 5.4 TB/s); for 12-bit ones (131072 x 16:
// 3.2 TB/s) no unit is busy: a stage's round (copy, restore, refill) over 16 stages an SM, about 49 KB, of
// which the products wait for K 45% of the time; for short prefixes a chain of about 8 us: group table, page
// ids, pages, scores, weights, output.
//
// Split: a unit is (group, KV head, tile of 128 or 256 rows); the units' blocks of 128 tokens are one
// line, cut into equal ranges, a CTA each, so that any mix of groups keeps all SMs busy.
#include <cuda.h>

#include <cstring>

#include "prefix.cuh"
#include "tc.cuh"

namespace kvz {

constexpr int kPfxPages = kPfxBlock / kPage;
constexpr uint32_t kUnitBytes = kPfxBlock * kDim * 2;  // K or V of a block, BF16
constexpr uint32_t kHalfBytes = kUnitBytes / 2;        // its 64-column halves
constexpr uint32_t kQTileBytes = 128 * kDim * 2;       // 128 query rows, BF16
constexpr uint32_t kQHalfBytes = kQTileBytes / 2;
constexpr uint32_t kGroupBytes = kPage * kDim * 2;  // most bytes of a coded (or raw) K or V group
constexpr int kInfoRing = 8;
// tensor memory, 256 columns a stream: 128 of scores, each 32 tokens' overwritten by their weights (16
// columns of high, 16 of low parts), the first 64 columns later by all tokens' third parts, and 128 of
// output
constexpr uint32_t kColO = 256;

// Two streams of softmax threads share a CTA.  kTiles = 2: 256 query rows, stream s holds rows
// [128 s, 128 s + 128) and both see every block.  kTiles = 1: 128 rows, the streams take
// alternate blocks and leave separate partials.
//
// Raw pages are copied by TMA into the operands' layout.  12-bit pages are copied as they are, a
// block's eight K groups and eight V groups into stages of their own, and restored by warps for K and
// for V: K of the next blocks is read and restored while V waits for room.  (Restored in place, without
// stages and with a third block in each ring, a 131072-token prefix x 16 sequences took 186 us against
// 143.)  The softmax threads take most registers: 168 a thread at launch (64512) become 256 x 208 +
// 128 x 80 = 63488 for raw pages.  For 12-bit pages and two weight parts, 96 (61440) become 256 x 136 +
// 384 x 64 = 59392, with a producer warp each for K and V and four restoring warps each (one producer
// and three restoring warps each: 148 us); three parts need more registers, 128 (65536) become 256 x 200
// + 256 x 56 = 65536.
template <int kFmt, int kTiles, int kParts>
struct PfxSmem {
    static constexpr bool coded = kFmt != kFmtRaw, many = coded && kParts == 2;
    static constexpr int threads = many ? 640 : coded ? 512 : 384;
    static constexpr int softmax_regs = many ? 136 : coded ? 200 : 208, other_regs = many ? 64 : coded ? 56 : 80;
    // 12-bit pages: producer warps (8 and, of two, 10), warps that restore K, as many for V behind them
    static constexpr int producers = many ? 2 : 1, restorers = many ? 4 : 3, restore0 = many ? 11 : 10;
    // rings of K blocks and of V blocks: K's are given back as soon as the scores are made, V's
    // when the weights have been used
    static constexpr int ku = kTiles == 2 ? (coded ? 1 : 2) : (coded ? 2 : 3), vu = coded ? 2 : 3, units = ku + vu;
    // operand layout: bytes from eight rows to the next, from 64 columns to the next
    static constexpr uint32_t rows8 = 1024, cols64 = kHalfBytes;
    static constexpr int stages = coded ? 2 * kPfxPages : 0;  // coded groups of a block
    __host__ __device__ static constexpr int slot(int n, int kv) { return kv ? ku + n % vu : n % ku; }
    __host__ __device__ static constexpr uint32_t phase(int n, int kv) { return (kv ? n / vu : n / ku) & 1; }
    static constexpr int arrivals = coded ? restorers : 1;  // that fill a block
    static constexpr int q = 0;
    static constexpr int ring = q + kTiles * (int)kQTileBytes;
    static constexpr int stage = ring + units * (int)kUnitBytes;
    static constexpr int full = stage + stages * (int)kGroupBytes;
    static constexpr int empty = full + units * 8;
    static constexpr int qfull = empty + units * 8;
    static constexpr int sfull = qfull + 8;    // [2] scores of a stream are in tensor memory
    static constexpr int pready = sfull + 16;  // [2][3] its weights of half a block are, third parts
    static constexpr int pused = pready + 48;  // [2] those of the first half have been used
    static constexpr int ofull = pused + 16;   // [2] its output of the segment is complete
    static constexpr int drain = ofull + 16;
    static constexpr int sarrived = drain + 8;  // [stages] coded groups
    static constexpr int sempty = sarrived + stages * 8;
    static constexpr int sinfo = sempty + stages * 8;
    static constexpr int info = sinfo + stages * 8;   // [kInfoRing][8] bad pages of a block
    static constexpr int misc = info + kInfoRing * 8;  // tensor memory address, abort flag, busy CTAs
    static constexpr int plan = misc + 16;  // [groups + 1] {first unit, first block}
    static int bytes(int groups) { return plan + (groups + 1) * 8; }
};

struct PfxSeg {
    int g, kvh, tile, unit, block0, blocks, len, seq0, rows;  // rows of this unit's tile
};

__device__ __forceinline__ PfxSeg pfx_locate(const PrefixParams &P, const int2 *plan, int x, int hi)
{
    int lo = 0, top = P.num_groups - 1;
    while (lo < top) {  // the last group that begins at or before x
        const int mid = (lo + top + 1) >> 1;
        if (plan[mid].y <= x) lo = mid;
        else top = mid - 1;
    }
    const PfxGroup r = pfx_group(P, lo);
    const int rem = x - plan[lo].y, ui = rem / r.blocks;
    PfxSeg s;
    s.g = lo;
    s.block0 = rem - ui * r.blocks;
    s.kvh = ui / r.tiles;
    s.tile = ui - s.kvh * r.tiles;
    s.unit = plan[lo].x + ui;
    s.blocks = min(hi - x, r.blocks - s.block0);
    s.len = r.len;
    s.seq0 = r.seq0;
    s.rows = min(r.seqs * P.G - s.tile * P.unit_rows, P.unit_rows);
    return s;
}

// A bounded wait that gives up for the whole CTA.
struct PfxWait {
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

// A K or V group in its stage: {kind | valid tokens of a raw one << 8, tags}.
enum : uint32_t { kGroupNone = 0, kGroupCoded = 1, kGroupRaw = 2, kGroupBad = 3 };

// A coded group (four blocks of 512 values) -> rows 16 page .. 16 page + 15 of an operand's block.
// A block's fragments are 8 x 8 matrices in the storage order's lanes: stmatrix puts their rows
// where the swizzled operand wants them (V's are dims x tokens and are stored back transposed).
// A group without raw blocks, the common one, has its blocks at fixed places: all loads are issued
// before any is used.  K and V share the code: the kernel's roles run side by side and their loops
// have to fit the instruction caches together (unrolled by role as well, a third of the stalls were
// for instructions).
__device__ __forceinline__ void pfx_restore_group(const uint8_t *src, uint32_t tags, uint32_t unit, int page, int lane,
                                                  bool is_v)
{
    const int mi = lane >> 3, rr = lane & 7;
    const int row = 16 * page + rr + 8 * (is_v ? mi >> 1 : mi & 1), c8 = is_v ? mi & 1 : mi >> 1;
    // 16-byte column 4 (j % 2) + 2 f + c8 of the rows of half j / 2, swizzled by the row
    const uint32_t at = unit + row * 128, col = (uint32_t)((c8 ^ rr) << 4);
    auto put = [&](uint32_t to, const uint32_t (&a)[4]) {
        if (is_v) stmatrix_x4_trans(to, a);
        else stmatrix_x4(to, a);
    };
    if (!(tags & 0x80808080u)) {
        uint4 low[4];
        uint2 code[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            low[j] = *reinterpret_cast<const uint4 *>(src + 768 * j + 16 * lane);
            code[j] = *reinterpret_cast<const uint2 *>(src + 768 * j + 512 + 8 * lane);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t bb = __byte_perm(tags, 0, 0x1111 * j);  // the block's tag in every byte
            const uint32_t to = at + (j >> 1) * kHalfBytes + (col ^ (64u * (j & 1)));
            uint32_t a[4];
            restore_fragment(low[j].x, low[j].y, code[j].x, bb, a);
            put(to, a);
            restore_fragment(low[j].z, low[j].w, code[j].y, bb, a);
            put(to ^ 32u, a);
        }
        return;
    }
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
        const bool raw = (tags & 0x80u) != 0;
        const uint8_t *lo = src + (raw ? 32 : 16) * lane, *hi = src + (raw ? 32 * lane + 16 : 512 + 8 * lane);
        const uint4 x = *reinterpret_cast<const uint4 *>(lo);
        const uint2 y = *reinterpret_cast<const uint2 *>(hi), z = raw ? *reinterpret_cast<const uint2 *>(hi + 8) : make_uint2(0, 0);
        uint32_t a[2][4] = {{x.x, x.y, x.z, x.w}, {y.x, y.y, z.x, z.y}};
        if (!raw) {
            const uint32_t bb = __byte_perm(tags, 0, 0x0000);
            restore_fragment(x.x, x.y, y.x, bb, a[0]);
            restore_fragment(x.z, x.w, y.y, bb, a[1]);
        }
        const uint32_t to = at + (j >> 1) * kHalfBytes + (col ^ (64u * (j & 1)));
        put(to, a[0]);
        put(to ^ 32u, a[1]);
        src += raw ? KVZ_BLOCK_BYTES_RAW : KVZ_BLOCK_BYTES_ELIGIBLE;
        tags >>= 8;
    }
}

// Eight flags as bytes and back.
__device__ __forceinline__ uint64_t spread_bits(uint32_t bits)
{
    uint64_t r = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) r |= (uint64_t)(bits >> i & 1) << (8 * i);
    return r;
}
__device__ __forceinline__ uint32_t gather_bits(uint64_t bytes) { return (uint32_t)((bytes * 0x0102040810204080ull) >> 56); }

template <int kFmt, int kTiles, int kParts>
__global__ void __launch_bounds__(PfxSmem<kFmt, kTiles, kParts>::threads, 1)
    k_prefix(const PrefixParams P, const __grid_constant__ CUtensorMap tmap)
{
    using S = PfxSmem<kFmt, kTiles, kParts>;
    constexpr bool kCoded = S::coded;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_addr(smem);
    if (sbase & 1023u) {  // swizzled operands need 1024-byte alignment
        if (threadIdx.x == 0) atomicOr(P.status, KVZ_STATUS_BAD_INDEX);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int2 *plan = reinterpret_cast<int2 *>(smem + S::plan);
    uint64_t *info = reinterpret_cast<uint64_t *>(smem + S::info);  // a byte per page
    volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(smem + S::misc);

    if (tid == 0) {
        for (int s = 0; s < S::units; ++s) {
            mbar_init(sbase + S::full + 8 * s, S::arrivals);
            mbar_init(sbase + S::empty + 8 * s, 1);
        }
        mbar_init(sbase + S::qfull, 256);
        for (int s = 0; s < 2; ++s) {
            mbar_init(sbase + S::sfull + 8 * s, 1);
            for (int i = 0; i < 3; ++i) mbar_init(sbase + S::pready + 24 * s + 8 * i, 128);
            mbar_init(sbase + S::pused + 8 * s, 1);
            mbar_init(sbase + S::ofull + 8 * s, 1);
        }
        mbar_init(sbase + S::drain, 1);
        if (kCoded)
            for (int s = 0; s < S::stages; ++s) {
                mbar_init(sbase + S::sarrived + 8 * s, 1);
                mbar_init(sbase + S::sempty + 8 * s, 1);
            }
        misc[1] = 0;
        fence_barrier_init();
    }
    // launched while the kernel before it ends: nothing that it wrote is read before this.  The own-pages
    // kernel may be placed from here on; it reads what was complete before this kernel
    pdl_wait_primary();
    pdl_launch_dependents();
    if (warp == 9) tmem_alloc(sbase + S::misc, 512);
    if (warp == 0) {  // units and blocks before each group
        bool ok = true;  // starts in order and in range
        const int per = (P.num_groups + 31) / 32;
        const int g0 = min(P.num_groups, lane * per), g1 = min(P.num_groups, g0 + per);
        int u = 0, w = 0, busy = 0;
        uint32_t bad = 0;
        for (int g = g0; g < g1; ++g) {
            const int start = P.group_start[g], end = P.group_start[g + 1], len = P.prefix_lens[g];
            const PfxGroup r = pfx_group(P, start, end, len);
            ok &= 0 <= start && start <= end && end <= P.batch;
            bad |= len != r.len;
            u += P.hkv * r.tiles;
            w += P.hkv * r.tiles * r.blocks;
            busy += P.hkv * r.tiles * pfx_unit_ctas(P, r.blocks);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
            if (lane == 0) atomicOr(P.status, KVZ_STATUS_BAD_ORDER);
            u = w = busy = 0;
            bad = 0;
        }
        busy = __reduce_add_sync(0xffffffffu, busy);
        if (lane == 0) misc[2] = (uint32_t)busy;
        if (bad) atomicOr(P.status, KVZ_STATUS_BAD_INDEX);
        int su = u, sw = w;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, su, off), b = __shfl_up_sync(0xffffffffu, sw, off);
            if (lane >= off) {
                su += a;
                sw += b;
            }
        }
        int ru = su - u, rw = sw - w;
        for (int g = g0; g < g1; ++g) {
            plan[g] = make_int2(ru, rw);
            if (!ok || g + 1 == g1) continue;
            const PfxGroup r = pfx_group(P, g);
            ru += P.hkv * r.tiles;
            rw += P.hkv * r.tiles * r.blocks;
        }
        if (lane == 31) plan[P.num_groups] = make_int2(su, sw);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    const int W = plan[P.num_groups].y, C = min((int)gridDim.x, (int)misc[2]), c = blockIdx.x;
    const int lo = c < C ? pfx_first(c, W, C) : 0, hi = c < C ? pfx_first(c + 1, W, C) : 0;
    PfxWait wait{P.status, misc + 1, true};

    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::other_regs));
    if ((warp == 8 || warp == 10) && !kCoded) {
        // =============================== producer ===============================
        // One lane per page, 32 pages (four blocks) at a time; the ids of the next four
        // blocks are fetched while these are copied.  (Calling pages into L2 four blocks ahead
        // made a 131072-token prefix 12% slower.)  Eight pages of 16 rows make a block's K (or V) operand: two
        // boxes a page, one per 64-column half.  One warp copies K, one V: a copy takes its issuing warp
        // about 100 clocks, and a block has 32 of them.
        prefetch_tensormap(&tmap);
        const int kv = warp == 8 ? 0 : 1;
        const uint64_t keep = l2_evict_last();
        const int pages = (hi - lo) * kPfxPages;
        auto prep = [&](int y) -> int {  // the page's first row in the raw pool, -1: none, -2: bad
            if (y >= pages) return -1;
            const PfxSeg s = pfx_locate(P, plan, lo + y / kPfxPages, hi);
            const int p = s.block0 * kPfxPages + y % kPfxPages;
            if (p * kPage >= s.len) return -1;
            const int32_t id = ld_keep_s32(P.prefix_ids + (int64_t)s.g * P.max_pages + p, keep);
            if (id < 0 || id >= P.num_raw_pages) return -2;
            return (id * P.hkv + s.kvh) * 32;
        };
        int cur = prep(lane), nxt = prep(32 + lane);
        bool ok = true;
        for (int base = 0; base < pages && ok; base += 32) {
            if (cur == -2) atomicOr(P.status, KVZ_STATUS_BAD_INDEX);
            const uint32_t good = __ballot_sync(0xffffffffu, cur >= 0), bad = __ballot_sync(0xffffffffu, cur == -2);
            const int nn = prep(base + 64 + lane);
            for (int i = 0; i < 32 / kPfxPages; ++i) {
                const int n = base / kPfxPages + i;  // block within the range
                if (n >= hi - lo) break;
                const uint32_t live = (good >> (kPfxPages * i)) & 0xFFu;
                const int row = __shfl_sync(0xffffffffu, cur, kPfxPages * i + ((lane >> 1) & 7));
                const int slot = S::slot(n, kv);
                const uint32_t fullbar = sbase + S::full + 8 * slot;
                ok = __all_sync(0xffffffffu, wait(sbase + S::empty + 8 * slot, S::phase(n, kv) ^ 1));
                if (!ok) break;
                if (lane == 0) {
                    if (kv == 0) info[n % kInfoRing] = spread_bits((bad >> (kPfxPages * i)) & 0xFFu);
                    if (live) mbar_arrive_expect_tx(fullbar, __popc(live) * (kPage * kDim * 2));
                    else mbar_arrive(fullbar);
                }
                __syncwarp();
                if (lane < 2 * kPfxPages && row >= 0) {
                    const uint32_t dst =
                        sbase + S::ring + slot * kUnitBytes + (lane & 1) * kHalfBytes + (lane >> 1) * (kPage * 128);
                    tensor_copy_2d_g2s(dst, &tmap, (lane & 1) * 64, row + kv * kPage, fullbar);
                }
            }
            cur = nxt;
            nxt = nn;
        }
        // never leave with copies in flight: every fill is waited for by the products; after a
        // wait that gave up, 1 ms (copies take microseconds)
        if (!ok) {
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 1000000) {}
        }
    } else if (warp == 8 || (S::producers == 2 && warp == 10)) {
        // ========================= producer, 12-bit pages =========================
        // Lane p copies the K group of every block's page p, lane 8 + p its V group (of two producers:
        // lane p of the second), each as soon as its stage is free.  Places and sizes are worked out by the whole warp, 32 pages (four
        // blocks) at a time, two batches on hand, and handed to the copying lanes by shuffles; the
        // metadata of the third batch and the ids of the fourth are fetched ahead.  (A lane working
        // out its own group while the others wait took 600 clocks a group.)
        const uint64_t keep = l2_evict_last();
        const int nb = hi - lo, page = lane & 7;
        const bool is_v = S::producers == 2 ? warp == 10 : (lane & 8) != 0, copies = lane < 2 * kPfxPages / S::producers;
        const int st = page + (is_v ? kPfxPages : 0);
        struct Pre {
            int32_t id;
            uint32_t what;  // KV head << 16 | valid tokens << 8 | kind
        };
        auto prep = [&](int y) -> Pre {
            if (y >= nb * kPfxPages) return Pre{-1, kGroupNone};
            const PfxSeg s = pfx_locate(P, plan, lo + y / kPfxPages, hi);
            const int p = s.block0 * kPfxPages + y % kPfxPages;
            if (p * kPage >= s.len) return Pre{-1, kGroupNone};
            const bool coded = p < s.len / kPage;  // the raw tail is the last page
            return Pre{coded ? ld_keep_s32(P.prefix_ids + (int64_t)s.g * P.max_pages + p, keep)
                             : ld_keep_s32(P.prefix_tail + s.g, keep),
                       (uint32_t)s.kvh << 16 | (uint32_t)min(kPage, s.len - p * kPage) << 8 |
                           (coded ? kGroupCoded : kGroupRaw)};
        };
        auto load_meta = [&](const Pre &r, uint64_t &mk, uint64_t &mv) {
            if ((r.what & 0xFFu) == kGroupCoded && r.id >= 0 && r.id < P.num_meta_pages)
                ld_keep_u64x2(P.meta + ((int64_t)r.id * P.hkv + (r.what >> 16)) * 2, keep, mk, mv);
        };
        struct Place {
            uint32_t what, offk, offv, tk, tv;  // raw: offk = index of the K and V pair
        };
        auto resolve = [&](const Pre &r, uint64_t mk, uint64_t mv) -> Place {
            Place q{r.what & 0xFFFFu, (uint32_t)mk, (uint32_t)mv, (uint32_t)(mk >> 32), (uint32_t)(mv >> 32)};
            uint32_t flag = 0;
            if ((q.what & 0xFFu) == kGroupCoded) {
                if (r.id < 0 || r.id >= P.num_meta_pages)
                    flag = KVZ_STATUS_BAD_INDEX;
                else if (!tags_valid(q.tk) || !tags_valid(q.tv) || q.offk == KVZ_OFFSET_INVALID || q.offv == KVZ_OFFSET_INVALID ||
                         ((uint64_t)q.offk + group_granules(q.tk)) * kGranule > P.arena_bytes ||
                         ((uint64_t)q.offv + group_granules(q.tv)) * kGranule > P.arena_bytes)
                    flag = KVZ_STATUS_BAD_META;
            } else if ((q.what & 0xFFu) == kGroupRaw) {
                if (r.id < 0 || r.id >= P.num_raw_pages) flag = r.id == -1 ? KVZ_STATUS_BAD_TAIL : KVZ_STATUS_BAD_INDEX;
                q.offk = (uint32_t)r.id * (uint32_t)P.hkv + (r.what >> 16);
            }
            if (flag) {
                q.what = kGroupBad;
                atomicOr(P.status, flag);
            }
            return q;
        };
        const Pre first = prep(lane), second = prep(32 + lane);
        Pre third = prep(64 + lane), fourth = prep(96 + lane);
        uint64_t mk[3] = {0, 0, 0}, mv[3] = {0, 0, 0};
        load_meta(first, mk[0], mv[0]);
        load_meta(second, mk[1], mv[1]);
        load_meta(third, mk[2], mv[2]);
        Place a = resolve(first, mk[0], mv[0]), b = resolve(second, mk[1], mv[1]);
        const uint32_t emptybar = sbase + S::sempty + 8 * st, bar = sbase + S::sarrived + 8 * st;
        uint64_t since = 0;
        bool ok = true;
        int batch = 0;  // of `a`
        for (int n = copies ? 0 : nb, idle = 0; ok && __any_sync(0xffffffffu, n < nb);) {
            const bool ready = n < nb && n / 4 <= batch + 1 && mbar_test_wait(emptybar, (n & 1) ^ 1);
            if (__any_sync(0xffffffffu, ready)) {
                const int from = 8 * (n & 3) + page;
                const bool later = n / 4 != batch;
                auto get = [&](uint32_t x, uint32_t y) {
                    const uint32_t u = __shfl_sync(0xffffffffu, x, from), v = __shfl_sync(0xffffffffu, y, from);
                    return later ? v : u;
                };
                const uint32_t what = get(a.what, b.what), offk = get(a.offk, b.offk), offv = get(a.offv, b.offv);
                const uint32_t tk = get(a.tk, b.tk), tv = get(a.tv, b.tv), kind = what & 0xFFu;
                if (ready) {
                    const uint32_t tags = is_v ? tv : tk;
                    *reinterpret_cast<uint2 *>(smem + S::sinfo + 8 * st) = make_uint2(what, tags);
                    if (kind == kGroupCoded) {
                        const uint32_t bytes = group_granules(tags) * kGranule;
                        mbar_arrive_expect_tx(bar, bytes);
                        bulk_copy_g2s(sbase + S::stage + st * kGroupBytes, P.arena + (uint64_t)(is_v ? offv : offk) * kGranule,
                                      bytes, bar);
                    } else if (kind == kGroupRaw) {
                        mbar_arrive_expect_tx(bar, kGroupBytes);
                        bulk_copy_g2s(sbase + S::stage + st * kGroupBytes,
                                      reinterpret_cast<const uint8_t *>(P.raw_pool) +
                                          ((uint64_t)offk * 2 + (is_v ? 1 : 0)) * kGroupBytes,
                                      kGroupBytes, bar);
                    } else {
                        mbar_arrive(bar);
                    }
                    ++n;
                }
                __syncwarp();
                idle = 0;
                if (__all_sync(0xffffffffu, n >= min(nb, 4 * (batch + 1)))) {  // every lane is done with `a`
                    ++batch;
                    a = b;
                    b = resolve(third, mk[2], mv[2]);
                    third = fourth;
                    load_meta(third, mk[2], mv[2]);
                    fourth = prep(32 * (batch + 3) + lane);
                }
            } else if ((++idle & 1023) == 0) {  // bounded: give up after kWaitLimitNs without a step
                const uint64_t now = globaltimer_ns();
                if (idle == 1024) since = now;
                if (misc[1] || now - since > kWaitLimitNs) {
                    if (lane == 0) atomicOr(P.status, KVZ_STATUS_TIMEOUT);
                    misc[1] = 1;
                    ok = false;
                }
                ok = __all_sync(0xffffffffu, ok);
            } else {
                __nanosleep(64);  // polling takes issue slots from the softmax warps of its scheduler
            }
        }
        if (!ok) {  // (as above: no copies in flight at the end)
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 1000000) {}
        }
    } else if (kCoded && warp >= S::restore0 && warp < S::restore0 + 2 * S::restorers) {
        // ================== 12-bit pages to BF16 operands ==================
        const bool is_v = warp >= S::restore0 + S::restorers;
        const int w = (warp - S::restore0) % S::restorers;
        bool ok = true;
        for (int n = 0; n < hi - lo && ok; ++n) {
            const int slot = S::slot(n, is_v);
            ok = __all_sync(0xffffffffu, wait(sbase + S::empty + 8 * slot, S::phase(n, is_v) ^ 1));
            const uint32_t unit = sbase + S::ring + slot * kUnitBytes;
            for (int page = w; page < kPfxPages && ok; page += S::restorers) {
                const int st = (is_v ? kPfxPages : 0) + page;
                const uint8_t *stage = smem + S::stage + st * kGroupBytes;
                ok = __all_sync(0xffffffffu, wait(sbase + S::sarrived + 8 * st, n & 1));
                if (!ok) break;
                const uint2 gi = *reinterpret_cast<const uint2 *>(smem + S::sinfo + 8 * st);
                const uint32_t kind = gi.x & 0xFFu;
                if (kind == kGroupCoded) {
                    pfx_restore_group(stage, gi.y, unit, page, lane, is_v);
                } else if (is_v || kind == kGroupRaw) {
                    // a raw tail as it is; rows of V without a token are zero, so that weight 0
                    // times them is 0 (scores of K rows without one are not used)
                    const uint32_t have = kind == kGroupRaw ? gi.x >> 8 : 0;
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) {
                        const int tok = 2 * i + (lane >> 4), ch = lane & 15, row = 16 * page + tok;
                        uint4 x = make_uint4(0, 0, 0, 0);
                        if ((uint32_t)tok < have) x = *reinterpret_cast<const uint4 *>(stage + tok * 256 + ch * 16);
                        *reinterpret_cast<uint4 *>(smem + S::ring + slot * kUnitBytes + (ch >> 3) * kHalfBytes + row * 128 +
                                                   (((ch & 7) ^ (row & 7)) << 4)) = x;
                    }
                }
                __syncwarp();
                if (lane == 0) {
                    if (!is_v) reinterpret_cast<uint8_t *>(info + n % kInfoRing)[page] = kind == kGroupBad;
                    mbar_arrive(sbase + S::sempty + 8 * st);
                }
            }
            fence_async_shared();
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(sbase + S::full + 8 * slot);
        }
    } else if (warp == 9) {
        // ============================ matrix products ============================
        // One warp issues for both streams in turn, which keeps them half a block apart: one
        // stream's softmax runs while the other's products do.  (A warp per stream let them fall
        // into step: 368 us against 313 for 128 x 8 heads over 65536 tokens.)
        constexpr uint32_t kQk = mma_desc(128, kPfxBlock, false), kPv = mma_desc(128, kDim, true);
        const uint32_t go = elect_one(), tm = uniform(tmem), sb = uniform(sbase);
        bool ok = true;
        auto wait_all = [&](uint32_t bar, uint32_t parity) {
            if (ok) ok = __all_sync(0xffffffffu, wait(bar, parity));
            tc_fence_after();
        };
        auto slot_of = [&](int n, int kv) { return uniform(S::slot(n, kv)); };
        auto wait_unit = [&](int n, int kv) { wait_all(sbase + S::full + 8 * S::slot(n, kv), S::phase(n, kv)); };
        // scores of stream s over K block n; give_back: the last product that reads the block
        auto qk = [&](uint32_t s, int n, bool give_back) {
            const uint32_t slot = slot_of(n, 0);
            const uint64_t a = smem_desc(sb + S::q + (kTiles == 2 ? s * kQTileBytes : 0), 16, 1024);
            const uint64_t b = smem_desc(sb + S::ring + slot * kUnitBytes, 16, S::rows8);
#pragma unroll
            for (int k = 0; k < 8; ++k)  // 16 of the 128 dims: 32 bytes within a half's rows
                mma_ss(go, tm + s * 128, a + (((k >> 2) * kQHalfBytes + (k & 3) * 32) >> 4),
                       b + (((k >> 2) * S::cols64 + (k & 3) * 32) >> 4), kQk, k > 0);
            mma_commit(go, sb + S::sfull + 8 * s);
            if (give_back) mma_commit(go, sb + S::empty + 8 * slot);
        };
        // output of stream s: its weights of 64 tokens (two parts of 32 tokens after two of the 32 before)
        // times half of the V block in slot
        auto pv = [&](uint32_t s, uint32_t slot, uint32_t half, bool add) {
            const uint64_t b = smem_desc(sb + S::ring + slot * kUnitBytes + half * 8 * S::rows8, S::cols64, S::rows8);
            const uint32_t w = tm + s * 128 + half * 64, o = tm + kColO + s * 128;
#pragma unroll
            for (int k = 0; k < 4; ++k)  // 16 tokens: two atoms of V rows, eight columns of weights
#pragma unroll
                for (int part = 0; part < 2; ++part)
                    mma_ts(go, o, w + (k >> 1) * 32 + part * 16 + (k & 1) * 8, b + ((k * 2 * S::rows8) >> 4), kPv,
                           part || k ? true : add);
            if (kParts == 3 && half == 0) mma_commit(go, sb + S::pused + 8 * s);
        };
        auto pv_third = [&](uint32_t s, uint32_t slot) {  // third parts, all 128 tokens
            const uint64_t b = smem_desc(sb + S::ring + slot * kUnitBytes, S::cols64, S::rows8);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                mma_ts(go, tm + kColO + s * 128, tm + s * 128 + k * 8, b + ((k * 2 * S::rows8) >> 4), kPv, true);
        };
        constexpr int step = kTiles == 2 ? 1 : 2;  // blocks between a stream's blocks
        uint32_t pphase = 0;                       // bit s
        int seg = 0;
        for (int x = lo; x < hi && ok; ++seg) {
            const PfxSeg sg = pfx_locate(P, plan, x, hi);
            const int n0 = x - lo, nb = sg.blocks;
            wait_all(sbase + S::qfull, seg & 1);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int j = kTiles == 2 ? 0 : s;
                if (j >= nb || !ok) break;
                if (kTiles == 1 || s == 0) wait_unit(n0 + j, 0);
                if (ok) qk(s, n0 + j, kTiles == 1 || s == 1);
            }
            for (int i = 0; i < (kTiles == 2 ? nb : (nb + 1) / 2) && ok; ++i) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {  // the streams in turn
                    const int j = kTiles == 2 ? i : 2 * i + s;
                    if (j >= nb || !ok) break;
                    const uint32_t ph = pphase >> s & 1, pbar = sbase + S::pready + 24 * s, slot = slot_of(n0 + j, 1);
                    if (kTiles == 1 || s == 0) wait_unit(n0 + j, 1);
                    wait_all(pbar, ph);
                    if (!ok) break;
                    pv(s, slot, 0, i % P.fold != 0);
                    if (j + step < nb && (kTiles == 1 || s == 0)) wait_unit(n0 + j + step, 0);
                    wait_all(pbar + 8, ph);
                    if (!ok) break;
                    pv(s, slot, 1, true);
                    if (kParts == 3) {
                        wait_all(pbar + 16, ph);
                        if (!ok) break;
                        pv_third(s, slot);
                    }
                    pphase ^= 1u << s;
                    if (j + step >= nb) mma_commit(go, sb + S::ofull + 8 * s);
                    if (kTiles == 1 || s == 1) mma_commit(go, sb + S::empty + 8 * slot);
                    if (j + step < nb) qk(s, n0 + j + step, kTiles == 1 || s == 1);
                }
            }
            x += nb;
        }
        if (!ok) {  // no product in flight when tensor memory is given back
            mma_commit(go, sbase + S::drain);
            mbar_wait(sbase + S::drain, 0, P.status);
        }
        __syncwarp();
    } else if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::softmax_regs));
        // ================================ softmax ================================
        // Thread = query row.  Its 128 scores of a block are read twice, for the maximum and, 64 tokens
        // at a time, for the weights, which go back over them: p = high + low in BF16, 16 bits of p
        // (off by at most 2^-17 of p, a 2^-9 part of a BF16 output's own rounding), and a third part,
        // all of p, for fp32 outputs.  The product with the first half of V runs while the second half is
        // made.  (All scores in registers and unrolled code: 155 K clocks for 27 blocks of 256 rows
        // against 143 K this way; the loops of all roles share the instruction caches.)  The
        // running maximum moves, and the output is rescaled, only when it grows by more than
        // 2^8: weights up to 2^8 lose nothing in floating point.  Every P.fold blocks the output
        // is added to the partial in memory and begins anew: the tensor cores' fp32 sums drop
        // the bits below the accumulator's last, a bias that grows with the steps of a sum.
        const int s = warp >> 2, quad = warp & 3, r = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t tS = tmem + s * 128 + lanes, tO = tmem + kColO + s * 128 + lanes;
        const uint64_t scale = pack2(P.scale_log2, P.scale_log2), minus = pack2(-1.f, -1.f);
        uint32_t sphase = 0, ophase = 0;
        for (int x = lo; x < hi;) {  // (after a wait that gave up, every segment's barriers still)
            const PfxSeg sg = pfx_locate(P, plan, x, hi);
            const int n0 = x - lo, nb = sg.blocks;
            // ---- queries to shared memory: sixteen threads a row; all loads in flight at once, and
            // before the barrier (behind it every product of the last segment is complete) ----
            const int ch = tid & 15;
            uint4 qv[8 * kTiles];
#pragma unroll
            for (int i = 0; i < 8 * kTiles; ++i) {
                const int row = (tid >> 4) + 16 * i, grow = sg.tile * P.unit_rows + row;
                qv[i] = make_uint4(0, 0, 0, 0);
                const int seq = P.G == 1 ? grow : (int)__umulhi(grow, P.over_G);
                if (row < sg.rows)
                    qv[i] = *reinterpret_cast<const uint4 *>(
                        P.q + ((int64_t)(sg.seq0 + seq) * P.hkv * P.G + sg.kvh * P.G + grow - seq * P.G) * kDim + ch * 8);
            }
            __syncwarp();
            asm volatile("bar.sync 1, 256;" ::: "memory");
#pragma unroll
            for (int i = 0; i < 8 * kTiles; ++i) {
                const int row = (tid >> 4) + 16 * i;
                *reinterpret_cast<uint4 *>(smem + S::q + (row >> 7) * kQTileBytes + (ch >> 3) * kQHalfBytes +
                                           (row & 127) * 128 + (((ch & 7) ^ (row & 7)) << 4)) = qv[i];
            }
            fence_async_shared();
            mbar_arrive(sbase + S::qfull);
            const int row0 = kTiles == 2 ? s * 128 : 0;
            const bool active = row0 + quad * 32 < sg.rows;  // a warp without rows only keeps step
            const int64_t slot0 = ((int64_t)(sg.unit + c) * 2 + s) * 128 + quad * 32;  // the warp's first row
            const int rows = min(32, sg.rows - row0 - quad * 32);
            float m = -INFINITY, l = 0.f;
            // The warp's 32 rows of output, complete in tensor memory and relative to maximum ref,
            // added to their partials, 32 columns at a time, each lane its row.  The partials of 32 rows are
            // laid out [8 columns][row], so that a store of the warp writes whole lines.
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
            for (int j = kTiles == 2 ? 0 : s; j < nb; j += kTiles == 2 ? 1 : 2, ++mine) {
                const int n = n0 + j;
                wait(sbase + S::sfull + 8 * s, sphase);
                sphase ^= 1;
                if (!__all_sync(0xffffffffu, wait.ok)) break;
                tc_fence_after();
                // (the products behind these scores were issued after every earlier product of the
                // stream, so its output is complete)
                const bool fresh = mine % P.fold == 0;  // the output begins anew
                if (fresh && mine > 0 && active) fold(m);
                const int left = sg.len - (sg.block0 + j) * kPfxBlock;
                const uint32_t bad = gather_bits(info[n % kInfoRing]);
                const bool whole = left >= kPfxBlock && bad == 0;
                if (!kCoded && !whole) {
                    // rows of V that hold no token: zero, so that weight 0 times them is 0
                    const int slot = S::slot(n, 1);
                    wait(sbase + S::full + 8 * slot, S::phase(n, 1));
                    if (r >= left || (bad >> (r >> 4) & 1)) {
                        uint8_t *at = smem + S::ring + slot * kUnitBytes + r * 128;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            *reinterpret_cast<uint4 *>(at + 16 * i) = make_uint4(0, 0, 0, 0);
                            *reinterpret_cast<uint4 *>(at + kHalfBytes + 16 * i) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    fence_async_shared();
                    if (!__all_sync(0xffffffffu, wait.ok)) break;
                }
                if (!whole && active) {  // scores without a token: minus infinity
#pragma unroll 1
                    for (int w = 0; w < 4; ++w) {
                        uint32_t live = left >= 32 * w + 32 ? ~0u : left <= 32 * w ? 0u : (1u << (left - 32 * w)) - 1;
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
                    const bool grow = mine == 0 || bm > m + 8.f;
                    if (mine > 0 && __any_sync(0xffffffffu, grow)) {
                        const float f = grow ? (m == -INFINITY ? 0.f : ex2(m - bm)) : 1.f;
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
                    if (grow) m = bm;
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
                                const uint64_t p = pack2(p0, p1);
                                sum[i & 1] = add2(sum[i & 1], p);
                                auto rest = [&](uint64_t x, uint32_t part) {  // x without its BF16 part, exact
                                    return fma2(pack2(__uint_as_float(part << 16), __uint_as_float(part & 0xFFFF0000u)), minus, x);
                                };
                                float r0, r1;
                                hi2[i] = pack_bf16x2(p0, p1);
                                const uint64_t r = rest(p, hi2[i]);
                                unpack2(r, r0, r1);
                                lo2[i] = pack_bf16x2(r0, r1);
                                if (kParts == 3) {
                                    unpack2(rest(r, lo2[i]), r0, r1);
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
            // ---- the segment's partial ----
            if (mine > 0) {
                wait(sbase + S::ofull + 8 * s, ophase);
                ophase ^= 1;
                tc_fence_after();
            }
            if (mine > 0 && active && __all_sync(0xffffffffu, wait.ok)) fold(m);
            tc_fence_before();
            if (lane < rows) *reinterpret_cast<float2 *>(P.part_ml + (slot0 + lane) * 2) = make_float2(m, l);
            x += nb;
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
// merge: one block per (sequence, KV head), one to eight of its eight warps per query head.  The
// partials of a head's row, the prefix's CTAs in order and then the own pages' CTAs in order, are
// dealt to the head's warps in turn; a warp takes 32 at a time (a lane each for the maxima and
// sums, all lanes for the outputs) into a running maximum, sum and output, and the warps of a head
// are added in order.
// ---------------------------------------------------------------------------------
constexpr int kMergeThreads = 256, kMergeWarps = kMergeThreads / 32;

__global__ void __launch_bounds__(kMergeThreads) k_prefix_merge(const PrefixParams P, const AttnParams A)
{
    __shared__ int red[kMergeWarps][3];
    __shared__ float2 wml[kMergeWarps];
    __shared__ float4 acc[kMergeWarps][32];
    const int b = blockIdx.x / P.hkv, kvh = blockIdx.x % P.hkv, tid = threadIdx.x;
    const int warp = tid >> 5, lane = tid & 31;
    // ---- before the wait: what the lengths say (they were complete before the call) ----
    int v[3] = {0, 0, 0};  // own pages of the sequences before b, of b, of all
    for (int i = tid; i < P.batch; i += kMergeThreads) {
        const int pages = (named_tokens(A.seq_lens[i], A.max_pages, A.tail_page != nullptr) + kPage - 1) / kPage;
        v[0] += i < b ? pages : 0;
        v[1] += i == b ? pages : 0;
        v[2] += pages;
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] = __reduce_add_sync(0xffffffffu, v[i]);
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < 3; ++i) red[warp][i] = v[i];
    }
    const PfxPlace where = pfx_place(P, b, lane);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        v[i] = 0;
#pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) v[i] += red[w][i];
    }
    const int share = P.G > 4 ? 1 : P.G > 2 ? 2 : P.G > 1 ? 4 : 8;  // warps of a head
    const int hg = warp / share, part = warp % share;
    PfxItems pre{0, 0, 0};
    if (hg < P.G) pre = pfx_items(P, where, b, kvh, hg);
    // own items: CTAs of the split kernel that hold pages of (b, kvh)
    const int64_t T = (int64_t)P.hkv * v[2], AC = A.grid;
    int ns = 0, a0 = 0;
    if (v[1] > 0 && hg < P.G) {
        const int64_t first = (int64_t)P.hkv * v[0] + (int64_t)kvh * v[1];
        a0 = (int)(first * AC / T);
        ns = (int)((first + v[1] - 1) * AC / T) - a0 + 1;
    }
    const int items = pre.n + ns, heads = P.G > 4 ? 8 : 4;  // heads: of a slot of the split kernel
    auto own_row = [&](int i) { return ((int64_t)(b * P.hkv + kvh) + a0 + i) * heads + hg; };
    pdl_wait_primary();  // both kernels' partials are complete
    RowSum sum;
    for (int i0 = part; i0 < items; i0 += 32 * share) {
        const int mine = i0 + lane * share;
        float2 e = make_float2(-INFINITY, 0.f);
        if (mine < items) {
            const int64_t cc = a0 + (mine - pre.n);
            // (a CTA of the split kernel without pages wrote nothing)
            if (mine < pre.n)
                e = *reinterpret_cast<const float2 *>(P.part_ml + (pre.first + (int64_t)mine * pre.step) * 2);
            else if (T >= AC || (cc * T + AC - 1) / AC < ((cc + 1) * T + AC - 1) / AC)
                e = *reinterpret_cast<const float2 *>(A.part_ml + own_row(mine - pre.n) * 2);
        }
        sum.add(e.x, e.y, [&](int k) {
            const int i = i0 + k * share;
            return i < pre.n ? *pfx_part(P, pre.first + (int64_t)i * pre.step, lane)
                             : reinterpret_cast<const float4 *>(A.part_o + own_row(i - pre.n) * kDim)[lane];
        });
    }
    if (share > 1) {
        acc[warp][lane] = sum.o;
        if (lane == 0) wml[warp] = make_float2(sum.m, sum.l);
        __syncthreads();
        if (part > 0) return;
        for (int k = 1; k < share; ++k) sum.add(wml[warp + k].x, wml[warp + k].y, acc[warp + k][lane]);
    }
    if (hg < P.G) sum.store(P, (int64_t)blockIdx.x * P.G + hg, lane);
}

// ---------------------------------------------------------------------------------
// launcher
// ---------------------------------------------------------------------------------
template <int kFmt, int kTiles, int kParts>
static cudaError_t launch_prefix_impl(const PrefixParams &P, const CUtensorMap &map, cudaStream_t stream)
{
    const int bytes = PfxSmem<kFmt, kTiles, kParts>::bytes(P.num_groups);
    // per process and device: the whole shared memory (an attribute of the function)
    static unsigned long long done = 0;  // bit per device ordinal < 64
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !(dev < 64 && (__atomic_load_n(&done, __ATOMIC_ACQUIRE) >> dev) & 1ull)) {
        e = cudaFuncSetAttribute(k_prefix<kFmt, kTiles, kParts>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e == cudaSuccess && dev < 64) __atomic_fetch_or(&done, 1ull << dev, __ATOMIC_ACQ_REL);
    }
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(P.grid);
    cfg.blockDim = dim3(PfxSmem<kFmt, kTiles, kParts>::threads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_prefix<kFmt, kTiles, kParts>, P, map);
}

template <int kFmt>
static cudaError_t launch_prefix_of(const PrefixParams &P, const CUtensorMap &map, cudaStream_t stream)
{
    if (P.unit_rows == 256)
        return P.out_bf16 ? launch_prefix_impl<kFmt, 2, 2>(P, map, stream) : launch_prefix_impl<kFmt, 2, 3>(P, map, stream);
    return P.out_bf16 ? launch_prefix_impl<kFmt, 1, 2>(P, map, stream) : launch_prefix_impl<kFmt, 1, 3>(P, map, stream);
}

cudaError_t launch_prefix(const PrefixParams &P, int format, const void *prefix_map, const AttnParams &A,
                          const void *own_map, int sms, cudaStream_t stream)
{
    const bool after = P.num_groups > 0 && P.grid > 0;
    if (after) {
        CUtensorMap map;
        memcpy(&map, prefix_map, sizeof map);
        const cudaError_t e = format == kFmtRaw ? launch_prefix_of<kFmtRaw>(P, map, stream) : launch_prefix_of<kFmtZf>(P, map, stream);
        if (e != cudaSuccess) return e;
    }
    // (P.direct: no prefix kernel ran, the own tokens' kernel reads the prefix)
    if (A.grid == 0) return launch_own(A, P, format, own_map, after, sms, stream);
    // (fp32 outputs: three weight parts here as well.  32 sequences x 32/8 heads behind 2055 tokens with 0 to
    // 4000 own ones: raw pages 60.5 -> 61.0 us, 12-bit 60.2 -> 62.1; off by 9.4e-7 with two parts, 8.7e-7)
    cudaError_t e = launch_attention_partials(A, format, own_map, !P.out_bf16, stream);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(P.batch * P.hkv);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_prefix_merge, P, A);
}

}  // namespace kvz
