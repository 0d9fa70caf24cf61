// append.cu -- write new tokens' keys and values into the raw pages of a paged cache, with
// the rotary position applied on the way, and rotate their queries for the attention call
// that follows.
//
// Mathematics, per rotary pair (a, b) of a head and its angle theta:
//     a' = m (a cos theta - b sin theta),  b' = m (a sin theta + b cos theta)
// in fp32, rounded once to BF16.  theta = position * frequency, where the position comes
// from the pair's axis.  A frequency is kept in turns as a 64-bit fixed-point fraction F:
// position * F modulo 2^64 is then the angle modulo one turn exactly (the wrap of integer
// multiplication), so far positions lose nothing; the top 32 bits go through sincospif, whose
// fp32 argument rounds them to 24: off by at most 2^-25 of half a turn, 9.4e-8 rad.
//
// Bound: memory.  (Hq + 2 Hkv) 256 bytes a token are read once and written once: 16381 tokens of 48
// heads in 64 to 67 us, 6.0 to 6.2 TB/s, 0.88 to 0.91 of the measured copy bandwidth; one decode token is a launch.
//
// Layout: a row is one head of one token, 256 bytes, handled by eight lanes: each holds two
// 16-byte vectors, eight whole rotary pairs in either pairing.  A block takes a run of
// consecutive rows (whole tokens as far as possible), computes the sines of the tokens it
// touches once into shared memory (<= kAppendTokens x 64 pairs, a lane's eight pairs of a row
// side by side with the other lanes': no bank is asked twice) and then streams its rows; the
// loads of a row do not wait for the sines.  Token and head of a row come from its number within
// the block, a division in 32 bits.
#include "kvz_device.cuh"
#include "kvz_internal.h"

namespace kvz {

constexpr int kAppendThreads = 256;
constexpr int kAppendRows = kAppendThreads / 8;  // rows a block handles at once
constexpr int kAppendTokens = 8;                 // tokens a block may touch
constexpr int kAppendResident = 3;               // blocks an SM holds

// cs: the first of the eight pairs' (cos, sin), the next ones eight further each
__device__ __forceinline__ void rotate8(uint4 &x, uint4 &y, const float2 *cs, bool neighbours)
{
    uint32_t *w0 = reinterpret_cast<uint32_t *>(&x), *w1 = reinterpret_cast<uint32_t *>(&y);
    if (neighbours) {  // pairs are (low, high) halves of each word
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t &w = i < 4 ? w0[i] : w1[i - 4];
            const float a = __uint_as_float(w << 16), b = __uint_as_float(w & 0xFFFF0000u);
            const float2 t = cs[8 * i];
            w = pack_bf16x2(a * t.x - b * t.y, a * t.y + b * t.x);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // pairs are (x element, y element)
        const float a0 = __uint_as_float(w0[i] << 16), a1 = __uint_as_float(w0[i] & 0xFFFF0000u);
        const float b0 = __uint_as_float(w1[i] << 16), b1 = __uint_as_float(w1[i] & 0xFFFF0000u);
        const float2 t0 = cs[16 * i], t1 = cs[16 * i + 8];
        w0[i] = pack_bf16x2(a0 * t0.x - b0 * t0.y, a1 * t1.x - b1 * t1.y);
        w1[i] = pack_bf16x2(a0 * t0.y + b0 * t0.x, a1 * t1.y + b1 * t1.x);
    }
}

__global__ void __launch_bounds__(kAppendThreads, kAppendResident) k_append(const AppendParams P)
{
    __shared__ float2 cs[kAppendTokens][64];
    const int H = P.hq + 2 * P.hkv, tid = threadIdx.x;
    const int64_t row0 = (int64_t)blockIdx.x * P.rows_per_block;
    const int64_t row1 = min(row0 + P.rows_per_block, (int64_t)P.tokens * H);
    const int tok0 = (int)(row0 / H), rows = (int)(row1 - row0);
    const uint32_t head0 = (uint32_t)(row0 - (int64_t)tok0 * H);
    const int toks = (int)((head0 + rows - 1) / (uint32_t)H) + 1;
    const int pairs = P.rot / 2;
    const int u = tid & 7;  // the lane's eight pairs (or 16 plain elements) of a row
    const bool turning = u < P.rot / 16;
    const int e0 = turning && !P.neighbours ? 8 * u : 16 * u;
    const int e1 = turning && !P.neighbours ? pairs + 8 * u : 16 * u + 8;

    struct Row {
        uint4 x, y;
        uint16_t *dst;
        int tok;
        bool rotated;
    };
    // a row's source and destination; its two vectors are loaded here
    auto load = [&](int row, Row &r) {
        r.dst = nullptr;
        if (row >= rows) return;
        const uint32_t in = (head0 + row) / (uint32_t)H;
        r.tok = tok0 + (int)in;
        const int h = (int)(head0 + row - in * (uint32_t)H);
        const uint16_t *src;
        if (h < P.hq) {
            src = P.q + r.tok * P.q_token + h * P.q_head;
            r.dst = P.q_out + ((int64_t)r.tok * P.hq + h) * kDim;
            r.rotated = true;
        } else {
            const bool is_v = h >= P.hq + P.hkv;
            const int kvh = h - P.hq - (is_v ? P.hkv : 0);
            const uint32_t slot = (uint32_t)P.slots[r.tok];
            if (slot > INT32_MAX || slot / kPage >= P.num_raw_pages) {
                if (slot != 0xFFFFFFFFu && u == 0) atomicOr(P.status, KVZ_STATUS_BAD_INDEX);
                return;  // -1: a padding token
            }
            src = is_v ? P.v + r.tok * P.v_token + kvh * P.v_head : P.k + r.tok * P.k_token + kvh * P.k_head;
            r.dst = P.raw_pool +
                    ((((int64_t)(slot / kPage) * P.hkv + kvh) * 2 + (is_v ? 1 : 0)) * kPage + slot % kPage) * kDim;
            r.rotated = !is_v;
        }
        r.x = __ldcs(reinterpret_cast<const uint4 *>(src + e0));
        r.y = __ldcs(reinterpret_cast<const uint4 *>(src + e1));
    };
    auto store = [&](Row &r) {
        if (!r.dst) return;
        if (r.rotated && turning) rotate8(r.x, r.y, &cs[r.tok - tok0][u], P.neighbours);
        uint4 *d0 = reinterpret_cast<uint4 *>(r.dst + e0), *d1 = reinterpret_cast<uint4 *>(r.dst + e1);
        if (P.streaming) {
            __stcs(d0, r.x);
            __stcs(d1, r.y);
        } else {
            *d0 = r.x;
            *d1 = r.y;
        }
    };

    pdl_wait_primary();  // launched while the kernel before it ends
    Row a, b;
    int row = tid >> 3;
    load(row, a);
    load(row + kAppendRows, b);
    if (pairs > 0) {
        for (int i = tid; i < toks * pairs; i += kAppendThreads) {
            const int t = i / pairs, p = i - t * pairs;
            const uint64_t turns = P.rope[2 * p], axis = P.rope[2 * p + 1];
            float s = 0.f, c = 1.f;
            if (axis < (uint64_t)P.axes) {
                const int64_t pos = P.positions[axis * P.tokens + tok0 + t];
                const int32_t top = (int32_t)(uint32_t)(((uint64_t)pos * turns) >> 32);
                sincospif((float)top * 4.656612873077393e-10f, &s, &c);  // 2^-31 half turns
            } else {
                atomicOr(P.status, KVZ_STATUS_BAD_INDEX);  // an axis without positions: not turned
            }
            cs[t][(p & 7) * 8 + (p >> 3)] = make_float2(c * P.scale, s * P.scale);
        }
        __syncthreads();
    }
    for (; row < rows; row += 2 * kAppendRows) {
        Row c, d;
        load(row + 2 * kAppendRows, c);
        load(row + 3 * kAppendRows, d);
        store(a);
        store(b);
        a = c;
        b = d;
    }
}

cudaError_t launch_append(AppendParams P, int sms, cudaStream_t stream)
{
    const int H = P.hq + 2 * P.hkv;
    const int64_t rows = (int64_t)P.tokens * H;
    // passes of a block: as few as let one wave hold all rows, at most eight (whole tokens share their
    // sines), and even, since a thread keeps two rows in flight (1021 tokens of 48 rows: 7.4 us with eight)
    int64_t passes = (rows + (int64_t)kAppendRows * kAppendResident * sms - 1) / ((int64_t)kAppendRows * kAppendResident * sms);
    passes = passes <= 1 ? 1 : passes >= 8 ? 8 : (passes + 1) & ~1ll;
    int64_t per = passes * kAppendRows;
    const int64_t most = (int64_t)(kAppendTokens - 2) * H + 1;  // touches at most kAppendTokens tokens
    if (per > most) per = most;
    P.rows_per_block = (int)per;
    // Rows that would fill half of the 129 MB L2 are written past it (201 MB: 69.9 -> 66.9 us, 151 MB:
    // 55.8 -> 52.7); fewer stay there for the attention call that reads them (29 MB, in a run of appends that
    // nothing reads: 11.8 us, streamed 11.5).
    P.streaming = rows * kDim * 2 > (64ll << 20);
    const int64_t blocks = (rows + per - 1) / per;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kAppendThreads);
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_append, P);
}

}  // namespace kvz
