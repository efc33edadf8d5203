// row_common.hpp -- pieces shared by the row operators (layer norm, MXFP4):
// element types, eight-element loads and stores of rows at any alignment,
// reductions over part of a wave, and the MXFP4 block.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "convimg.h"

namespace convimg {

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32v4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

// A row may start at any element (odd widths, views into wider buffers), so
// a vector access is only as aligned as an element.  Global memory serves
// 16-byte accesses at any such address on gfx950, so these types let the
// compiler issue them.
typedef u32v4_t u32v4_a2_t __attribute__((aligned(2)));
typedef u32v4_t u32v4_a4_t __attribute__((aligned(4)));

struct Bf16 {
    typedef unsigned short raw;
    static constexpr int code = CONVIMG_BF16;
};
struct Fp16 {
    typedef unsigned short raw;
    static constexpr int code = CONVIMG_FP16;
};
struct Fp32 {
    typedef float raw;
    static constexpr int code = CONVIMG_FP32;
};
struct Mx4 {};      // packed MXFP4 rows

inline size_t dtype_bytes(int dtype) { return dtype == CONVIMG_FP32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == CONVIMG_BF16 || dtype == CONVIMG_FP16 || dtype == CONVIMG_FP32; }

// fp32 -> bf16, round to nearest, ties to even (one instruction for a pair).
__device__ __forceinline__ unsigned pack_bf16(float a, float b)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(unsigned, v);
}

__device__ __forceinline__ unsigned pack_fp16(float a, float b)
{
    const f16x2_t v = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(unsigned, v);
}

template <typename T>
__device__ __forceinline__ float load1(const typename T::raw *p)
{
    if constexpr (T::code == CONVIMG_FP32)
        return *p;
    else if constexpr (T::code == CONVIMG_BF16)
        return __uint_as_float((unsigned)*p << 16);
    else
        return (float)__builtin_bit_cast(_Float16, *p);
}

template <typename T>
__device__ __forceinline__ void store1(typename T::raw *p, float v)
{
    if constexpr (T::code == CONVIMG_FP32)
        *p = v;
    else if constexpr (T::code == CONVIMG_BF16)
        *p = (unsigned short)pack_bf16(v, 0.f);
    else
        *p = __builtin_bit_cast(unsigned short, (_Float16)v);
}

// Eight consecutive elements of a row as they lie in memory.
template <typename T>
struct Raw8 {
    u32v4_t w[T::code == CONVIMG_FP32 ? 2 : 1];
};

// Loads the eight from element `col` of a row of `cols`.  At the end of the
// row, the row's last eight elements instead, which keeps the load whole (a
// lane that loads single elements waits for them, and so for everything that
// the wave has in flight); tail8 moves them into place when they are used.
// Nothing is loaded past the row.  SHORT: rows may have fewer than eight.
template <typename T, bool SHORT = true>
__device__ __forceinline__ Raw8<T> load_raw8(const typename T::raw *row, int col, int cols)
{
    Raw8<T> r = {};
    if (!SHORT || cols >= 8) {
        if (col < cols) {
            const typename T::raw *p = row + min(col, cols - 8);
            if constexpr (T::code == CONVIMG_FP32) {
                r.w[0] = ((const u32v4_a4_t *)p)[0];
                r.w[1] = ((const u32v4_a4_t *)p)[1];
            } else {
                r.w[0] = *(const u32v4_a2_t *)p;
            }
        }
        return r;
    }
    typename T::raw e[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        e[k] = 0;
        if (col + k < cols)
            e[k] = row[col + k];
    }
    __builtin_memcpy(&r, e, sizeof(r));
    return r;
}

// What load_raw8 loaded, element `col` first and zeros past the row.
template <typename T, bool SHORT = true>
__device__ __forceinline__ Raw8<T> tail8(Raw8<T> r, int col, int cols)
{
    if ((cols & 7) == 0 || (SHORT && cols < 8))
        return r;
    const int past = col < cols ? max(col + 8 - cols, 0) : 0;      // elements to move down by
    constexpr int W = sizeof(r) / 4;
    unsigned w[W + 1];
    w[W] = 0;
    __builtin_memcpy(w, &r, sizeof(r));
    // (by 4, 2 and 1 elements; for 16-bit types 2, 1 and half a word)
#pragma unroll
    for (int e = 4; e >= 1; e >>= 1) {
        const bool on = (past & e) != 0;
        const int n = e * W / 8;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const unsigned v = n > 0 ? (i + n < W ? w[i + n] : 0u) : (w[i] >> 16) | (w[i + 1] << 16);
            w[i] = on ? v : w[i];
        }
    }
    __builtin_memcpy(&r, w, sizeof(r));
    return r;
}

template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T> &r, float (&v)[8])
{
    if constexpr (T::code == CONVIMG_FP32) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = __uint_as_float(r.w[e / 4][e % 4]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const unsigned w = r.w[0][e];
            if constexpr (T::code == CONVIMG_BF16) {
                v[2 * e] = __uint_as_float(w << 16);
                v[2 * e + 1] = __uint_as_float(w & 0xffff0000u);
            } else {
                const f16x2_t h = __builtin_bit_cast(f16x2_t, w);
                v[2 * e] = (float)h[0];
                v[2 * e + 1] = (float)h[1];
            }
        }
    }
}

template <typename T, bool SHORT = true>
__device__ __forceinline__ void load8(const typename T::raw *row, int col, int cols, float (&v)[8])
{
    unpack8<T>(tail8<T, SHORT>(load_raw8<T, SHORT>(row, col, cols), col, cols), v);
}

template <typename T>
__device__ __forceinline__ void store8(typename T::raw *row, int col, int cols, const float (&v)[8])
{
    if (col + 8 <= cols) {
        if constexpr (T::code == CONVIMG_FP32) {
            u32v4_t a, b;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[e] = __float_as_uint(v[e]);
                b[e] = __float_as_uint(v[4 + e]);
            }
            u32v4_a4_t *p = (u32v4_a4_t *)(row + col);
            p[0] = a;
            p[1] = b;
        } else {
            u32v4_t a;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                a[e] = T::code == CONVIMG_BF16 ? pack_bf16(v[2 * e], v[2 * e + 1])
                                               : pack_fp16(v[2 * e], v[2 * e + 1]);
            *(u32v4_a2_t *)(row + col) = a;
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (col + e < cols)
            store1<T>(row + col + e, v[e]);
}

// gfx950's swap of v's upper with its lower group of O lanes (O 16 or 32), in
// every pair of groups: element 0 holds the lower group's values in both
// groups of a pair, element 1 the upper group's.
template <int O>
__device__ __forceinline__ void lane_pair(float v, float (&r)[2])
{
    typedef unsigned u32v2 __attribute__((ext_vector_type(2)));
    const unsigned i = __float_as_uint(v);
    u32v2 s;
    if constexpr (O == 16)
        s = __builtin_amdgcn_permlane16_swap(i, i, false, false);
    else
        s = __builtin_amdgcn_permlane32_swap(i, i, false, false);
    r[0] = __uint_as_float(s[0]);
    r[1] = __uint_as_float(s[1]);
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v)
{
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}

// v plus the value O lanes away (in the lane number's bit O), for powers of
// two.  MIRROR: groups of O lanes hold one value each, so that a mirrored
// lane will do for O = 4 and 8.
template <int O, bool MIRROR>
__device__ __forceinline__ float pair_sum(float v)
{
    if constexpr (O == 1)
        return v + dpp<0xB1>(v);       // quad [1, 0, 3, 2]
    else if constexpr (O == 2)
        return v + dpp<0x4E>(v);       // quad [2, 3, 0, 1]
    else if constexpr (O == 4 && MIRROR)
        return v + dpp<0x141>(v);      // half row mirrored
    else if constexpr (O == 8)
        return v + dpp<MIRROR ? 0x140 : 0x128>(v);      // row mirrored, row rotated by 8
    else if constexpr (O == 4)
        return v + __shfl_xor(v, 4, 64);
    float r[2];
    lane_pair<O>(v, r);
    return r[0] + r[1];
}

// Sum over groups of W neighbouring lanes (W a power of two up to 64), the
// same in every lane of a group.
template <int W>
__device__ __forceinline__ float group_sum(float v)
{
    if constexpr (W >= 2)
        v = pair_sum<1, true>(v);
    if constexpr (W >= 4)
        v = pair_sum<2, true>(v);
    if constexpr (W >= 8)
        v = pair_sum<4, true>(v);
    if constexpr (W >= 16)
        v = pair_sum<8, true>(v);
    if constexpr (W >= 32)
        v = pair_sum<16, true>(v);
    if constexpr (W >= 64)
        v = pair_sum<32, true>(v);
    return v;
}

// Sum over the lanes of a wave that are equal modulo W.
template <int W>
__device__ __forceinline__ float stride_sum(float v)
{
    if constexpr (W <= 4)
        v = pair_sum<4, false>(v);
    if constexpr (W <= 8)
        v = pair_sum<8, false>(v);
    if constexpr (W <= 16)
        v = pair_sum<16, false>(v);
    if constexpr (W <= 32)
        v = pair_sum<32, false>(v);
    return v;
}

// Largest of the four lanes of a quad.
__device__ __forceinline__ unsigned quad_max(unsigned v)
{
    v = max(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xf, 0xf, true));
    return max(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xf, 0xf, true));
}

// The MXFP4 scale byte of a block from the bits of its largest magnitude:
// floor(log2) is the exponent field, 2 the exponent of the grid's largest
// value (6 = 1.5 * 2^2).  Blocks below 2^-125 take the smallest scale,
// 2^-127; a block that holds an infinity or a NaN has no scale and takes
// 255, which stands for NaN.
__device__ __forceinline__ unsigned mx_scale_byte(unsigned top_bits)
{
    const int e = (int)(top_bits >> 23);
    return e == 255 ? 255u : (unsigned)(e > 2 ? e - 2 : 0);
}

// The scale dword of 128 columns (four blocks) that W / 4 quads of lanes hold,
// W 4, 8 or 16; `byte` is the scale byte of the lane's block `blk`.  All W
// lanes take part and get it.
template <int W>
__device__ __forceinline__ unsigned mx_scale_word(unsigned byte, int blk)
{
    unsigned w = byte << (8 * (blk & 3));
    if constexpr (W >= 8)
        w |= (unsigned)__builtin_amdgcn_mov_dpp((int)w, 0x141, 0xf, 0xf, true);      // half row mirrored
    if constexpr (W >= 16)
        w |= (unsigned)__builtin_amdgcn_mov_dpp((int)w, 0x140, 0xf, 0xf, true);      // row mirrored
    return w;
}

// 2^(byte - 127) for bytes 0 .. 254, NaN for 255: the fp32 exponent field,
// with 2^-127 a subnormal.
__device__ __forceinline__ float mx_scale_value(unsigned byte)
{
    return __uint_as_float(byte == 255u ? 0x7fc00000u : byte != 0 ? byte << 23 : 0x00400000u);
}

// Eight values over the scale, rounded to the nearest e2m1 (ties to even,
// saturating at 6), element 0 in the lowest nibble.
__device__ __forceinline__ unsigned mx_encode8(const float (&v)[8], float scale)
{
    unsigned r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], scale, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], scale, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], scale, 3);
    return r;
}

__device__ __forceinline__ void mx_decode8(unsigned codes, float scale, float (&v)[8])
{
    const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 0);
    const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 1);
    const f32x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 2);
    const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 3);
    v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1];
    v[4] = c[0]; v[5] = c[1]; v[6] = d[0]; v[7] = d[1];
}

// Bits of the larger magnitude of v and top (NaN and infinity above every
// finite value), as whole numbers.
__device__ __forceinline__ unsigned mx_top(unsigned top, float v)
{
    const unsigned m = __float_as_uint(v) & 0x7fffffffu;
    return m > top ? m : top;
}

// Rows and columns at most.  Kernels count a row's columns in an int and step
// up to 8192 past its end.
constexpr long long kMaxRows = 0x7fffffffLL, kMaxCols = 0x7fffffffLL - 0x3fff;

__host__ __device__ inline int mx_blocks(int cols) { return (cols + 31) / 32; }
inline int mx_quads(int cols) { return (cols + 127) / 128; }
inline size_t mx_code_bytes(long long rows, int cols) { return (size_t)rows * mx_blocks(cols) * 16; }
inline size_t mx_scale_bytes(long long rows, int cols) { return (size_t)rows * mx_quads(cols) * 4; }

// Rows and columns of a packed operand: its codes stay below 2^31 bytes.
inline int mx_shape(long long rows, long long cols)
{
    if (rows < 0 || cols <= 0)
        return CONVIMG_ERR_SHAPE;
    if (rows > kMaxRows || cols > kMaxCols || mx_code_bytes(rows, (int)cols) >= 0x80000000u)
        return CONVIMG_ERR_RANGE;
    return CONVIMG_OK;
}

inline bool row_overlaps(const void *a, size_t na, const void *b, size_t nb)
{
    if (!a || !b || !na || !nb)
        return false;
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + nb && y < x + na;
}

// Bytes from the first to the last element of `rows` rows of `cols` that
// start `ld` elements apart.
inline size_t span_bytes(long long rows, long long ld, int cols, int dtype)
{
    return rows <= 0 ? 0 : ((size_t)(rows - 1) * (size_t)ld + (size_t)cols) * dtype_bytes(dtype);
}

// Calls f with a value of the type that `dtype` names.
template <typename F>
inline void with_dtype(int dtype, F &&f)
{
    if (dtype == CONVIMG_BF16)
        f(Bf16{});
    else if (dtype == CONVIMG_FP16)
        f(Fp16{});
    else
        f(Fp32{});
}

}  // namespace convimg
