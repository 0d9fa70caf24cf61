// frags.cuh -- m16n8k16 A operands of a 16-token page in shared memory: 12-bit groups in storage
// order and plain BF16 pages loaded with the 128-byte swizzle.
#pragma once

#include "kvz_device.cuh"

namespace kvz {

__device__ __forceinline__ uint32_t swz128(int row, int col)
{
    // byte offset of element (row, col) of a [32][128] BF16 tile loaded as two
    // 64-column boxes with the 128-byte swizzle (16-byte chunk index ^= row % 8)
    return (uint32_t)((col >> 6) * 4096 + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4) + (col & 7) * 2);
}

// ---------------------------------------------------------------------------------
// consumer-side fragment loads
// ---------------------------------------------------------------------------------
// One 512-value block of a compressed group in shared memory -> the two A fragments.
__device__ __forceinline__ void block_frags(const uint8_t *blk, uint32_t tag, int lane, uint32_t (&a0)[4],
                                            uint32_t (&a1)[4])
{
    if (tag == 0xFFu) {
        const uint4 x = *reinterpret_cast<const uint4 *>(blk + 32 * lane);
        const uint4 y = *reinterpret_cast<const uint4 *>(blk + 32 * lane + 16);
        a0[0] = x.x; a0[1] = x.y; a0[2] = x.z; a0[3] = x.w;
        a1[0] = y.x; a1[1] = y.y; a1[2] = y.z; a1[3] = y.w;
    } else {
        const uint4 low = *reinterpret_cast<const uint4 *>(blk + 16 * lane);
        const uint2 code = *reinterpret_cast<const uint2 *>(blk + 512 + 8 * lane);
        const uint32_t bb = tag * 0x01010101u;
        restore_fragment(low.x, low.y, code.x, bb, a0);
        restore_fragment(low.z, low.w, code.y, bb, a1);
    }
}

// K operand (tokens x 16 dims) of k-tile (j, f) from a swizzled raw page.
__device__ __forceinline__ void raw_k_frag(uint32_t st, int j, int f, int lane, uint32_t (&a)[4])
{
    const int mi = lane >> 3, rr = lane & 7;
    const int tok = rr + 8 * (mi & 1), col = 32 * j + 16 * f + 8 * (mi >> 1);
    ldmatrix_x4(st + swz128(tok, col), a);
}

// V^T operand (16 dims x tokens) of tile (j, f) from a swizzled raw page.
__device__ __forceinline__ void raw_v_frag(uint32_t st, int j, int f, int lane, uint32_t (&a)[4])
{
    const int mi = lane >> 3, rr = lane & 7;
    const int tok = rr + 8 * (mi >> 1), col = 32 * j + 16 * f + 8 * (mi & 1);
    ldmatrix_x4_trans(st + swz128(16 + tok, col), a);
}

// Zero the V^T operand halves of tokens >= valid (a partial tail page may hold stale
// values beyond its last token; P is 0 there but 0 * NaN is not 0).
__device__ __forceinline__ void mask_v_frag(uint32_t (&a)[4], int lane, int valid)
{
    const int t = lane & 3;
    const int t0 = 2 * t, t1 = 2 * t + 1, t8 = 2 * t + 8, t9 = 2 * t + 9;
    const uint32_t mlo = (t0 < valid ? 0x0000FFFFu : 0u) | (t1 < valid ? 0xFFFF0000u : 0u);
    const uint32_t mhi = (t8 < valid ? 0x0000FFFFu : 0u) | (t9 < valid ? 0xFFFF0000u : 0u);
    a[0] &= mlo;
    a[1] &= mlo;
    a[2] &= mhi;
    a[3] &= mhi;
}

}  // namespace kvz
