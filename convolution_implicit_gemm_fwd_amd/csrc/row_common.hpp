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

// Eight consecutive elements of a row whose first is element `col`, of which
// those below `cols` exist; the others read as 0.
template <typename T>
__device__ __forceinline__ void load8(const typename T::raw *row, int col, int cols, float (&v)[8])
{
    if (col + 8 <= cols) {
        if constexpr (T::code == CONVIMG_FP32) {
            const u32v4_a4_t *p = (const u32v4_a4_t *)(row + col);
            const u32v4_t a = p[0], b = p[1];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = __uint_as_float(a[e]);
                v[4 + e] = __uint_as_float(b[e]);
            }
        } else {
            const u32v4_t a = *(const u32v4_a2_t *)(row + col);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const unsigned w = a[e];
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
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = col + e < cols ? load1<T>(row + col + e) : 0.f;
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

// Sum over groups of W neighbouring lanes (W a power of two up to 64), the
// same in every lane of a group.
template <int W>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1)
        v += __shfl_xor(v, o, 64);
    return v;
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

__host__ __device__ inline int mx_blocks(int cols) { return (cols + 31) / 32; }
inline int mx_quads(int cols) { return (cols + 127) / 128; }
inline size_t mx_code_bytes(long long rows, int cols) { return (size_t)rows * mx_blocks(cols) * 16; }
inline size_t mx_scale_bytes(long long rows, int cols) { return (size_t)rows * mx_quads(cols) * 4; }

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
