// mxint8.hpp -- microscaled 8-bit integers (MXINT8), the form in which
// activations are kept for the backward pass.
//
// A block is 32 consecutive values of a row.  Its unit is u = 2^(s - 127), s
// the smallest whole number of at least 1 for which 127 u reaches the block's
// largest magnitude, and a value is stored as value / u rounded to the nearest
// whole number, ties to even.  Nothing saturates, so a value is off by at most
// u / 2, and code * u has at most seven significant bits: exact in bf16.
#pragma once

#include "row_common.hpp"

namespace convimg {

inline size_t mxi_code_bytes(long long rows, int cols) { return (size_t)rows * mx_blocks(cols) * 32; }
inline size_t mxi_scale_bytes(long long rows, int cols) { return (size_t)rows * mx_quads(cols) * 4; }

// The scale byte from the bits of the block's largest magnitude: with e its
// exponent field 127 units of 2^(e - 6 - 127) reach it if its mantissa is at
// most 127 / 64, else those of twice the size do; the sum carries into the
// field in that case.  255 (NaN) for a block with an infinity or a NaN.
__device__ __forceinline__ unsigned mxi_scale_byte(unsigned top_bits)
{
    const int s = (int)((top_bits + 0x1ffffu) >> 23) - 6;
    return top_bits >= 0x7f800000u ? 255u : (unsigned)max(s, 1);
}

// Eight values over the unit as bytes.  v / u is exact; adding 1.5 * 2^23
// rounds it to a whole number, whose low byte is the sum's.
__device__ __forceinline__ uint2 mxi_encode8(const float (&v)[8], unsigned byte)
{
    if (byte == 255u)
        return uint2{0, 0};
    const float inv = __uint_as_float((254u - byte) << 23);
    unsigned t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        t[e] = __float_as_uint(__builtin_fmaf(v[e], inv, 12582912.f));
    return uint2{__builtin_amdgcn_perm(t[1], t[0], 0x0c0c0400u) | __builtin_amdgcn_perm(t[3], t[2], 0x04000c0cu),
                 __builtin_amdgcn_perm(t[5], t[4], 0x0c0c0400u) | __builtin_amdgcn_perm(t[7], t[6], 0x04000c0cu)};
}

__device__ __forceinline__ void mxi_decode8(uint2 c, float unit, float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = (float)(signed char)(c.x >> (8 * e)) * unit;
        v[4 + e] = (float)(signed char)(c.y >> (8 * e)) * unit;
    }
}

// Writes eight values of a row from column `col` on, zeros past its end, and
// the row's scale dwords, one a run of 128 columns.  A block is held by four
// neighbouring lanes and a dword's blocks by W lanes (mx_scale_word), which all
// reach this together.
template <int W>
__device__ __forceinline__ void mxi_emit8(unsigned char *codes, unsigned *scales, long long row, int cols, int col,
                                          const float (&v)[8])
{
    unsigned top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        top = mx_top(top, v[e]);
    const int kp = (cols + 31) & ~31;
    const unsigned byte = mxi_scale_byte(quad_max(top));
    if (col < kp)
        *(uint2 *)(codes + row * kp + col) = mxi_encode8(v, byte);
    const unsigned word = mx_scale_word<W>(col < kp ? byte : 0u, col >> 5);
    if ((col & 127) == 0 && col < kp)
        scales[row * ((cols + 127) >> 7) + (col >> 7)] = word;
}

// The unit of a column of a row.
__device__ __forceinline__ float mxi_unit(const unsigned char *scales, long long row, int cols, int col)
{
    return mx_scale_value(scales[row * (((cols + 127) >> 7) * 4) + (col >> 5)]);
}

}  // namespace convimg
