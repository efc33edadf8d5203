// adapter_expand.hpp -- the second half of low-rank adapters inside a product:
// adds scale_g h[m] up_g to the sums of a tile whose rows m may belong to
// different adapters g.
//
// Values are split into bf16 terms that add up to them exactly (bf16 1, fp16 2,
// fp32 3 terms of at most 8 bits), so that bf16 matrix instructions give fp32
// products: those of terms i and j with i + j <= 2, the others are below
// 2^-24 of the product.
#pragma once

#include "row_common.hpp"

namespace convimg {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

template <typename T>
constexpr int split_terms() { return T::code == CONVIMG_BF16 ? 1 : T::code == CONVIMG_FP16 ? 2 : 3; }

// Eight values as N bf16 terms, each the upper half of what is left.  An
// infinity is its own first term and leaves 0.
template <int N>
__device__ __forceinline__ void split8(const float (&v)[8], u32v4_t (&t)[N])
{
    unsigned w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        w[e] = __float_as_uint(v[e]);
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            t[n][e] = __builtin_amdgcn_perm(w[2 * e + 1], w[2 * e], 0x07060302u);
        if (n + 1 < N)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float a = __uint_as_float(w[e]), hi = __uint_as_float(w[e] & 0xffff0000u);
                w[e] = __float_as_uint(n == 0 && a == hi ? 0.f : a - hi);
            }
    }
}

// The terms of eight loaded values.
template <typename T>
__device__ __forceinline__ void split_raw8(const Raw8<T> &r, u32v4_t (&t)[split_terms<T>()])
{
    if constexpr (T::code == CONVIMG_BF16) {
        t[0] = r.w[0];
    } else {
        float v[8];
        unpack8<T>(r, v);
        split8(v, t);
    }
}

// c plus the product of two operands in terms, the small ones first.
template <int NA, int NB>
__device__ __forceinline__ f32x4_t mfma_terms16(const u32v4_t (&a)[NA], const u32v4_t (&b)[NB], f32x4_t c)
{
#pragma unroll
    for (int s = 2; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB)
                c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a[i]),
                                                            __builtin_bit_cast(bf16x8_t, b[s - i]), c, 0, 0, 0);
    return c;
}

template <int NA, int NB>
__device__ __forceinline__ f32x16_t mfma_terms32(const u32v4_t (&a)[NA], const u32v4_t (&b)[NB], f32x16_t c)
{
#pragma unroll
    for (int s = 2; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB)
                c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a[i]),
                                                            __builtin_bit_cast(bf16x8_t, b[s - i]), c, 0, 0, 0);
    return c;
}

struct MxNoAdapters {};

struct MxAdapterArgs {
    const float *h;        // [splits][M][r], to be summed over the splits
    const void *up;        // [G][r][N] in `dtype`
    const float *scale;    // [G]
    const int *ids;        // [M]
    int G, r, splits, dtype;
};

// h of a row from rank i0 on, eight values times s, zeros past the rank.
__device__ __forceinline__ void adapter_h8(const MxAdapterArgs &a, int M, int m, int i0, float s, float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = 0.f;
    for (int k = 0; k < a.splits; ++k) {
        const float *p = a.h + ((long long)k * M + m) * a.r;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (i0 + e < a.r)
                v[e] += p[i0 + e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] *= s;
}

// The sums of FM x FN blocks of 32 x 32 from row m0 and column n0 on; a lane
// holds row lane % 32 of a block and 16 of its columns (the instruction's rows).
//
// The wave goes through the adapters that its rows have, in the order of their
// first rows, so the tile costs one round of small loads and 3 FN FM matrix
// instructions a 16 ranks and adapter.  A row takes only its own adapter's
// product (selected after the product: a zero times another adapter's infinity
// would not do).
template <int FM, int FN>
__device__ __forceinline__ void adapter_expand(const MxAdapterArgs &a, int M, int N, int m0, int n0,
                                               f32x16_t (&acc)[FM][FN])
{
    const int lane = threadIdx.x & 63, half = lane >> 5, l32 = lane & 31;
    int id[FM];
    unsigned left[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int m = m0 + i * 32 + l32;
        id[i] = m < M ? a.ids[m] : -1;
        left[i] = (unsigned)__ballot(id[i] >= 0 && id[i] < a.G);
    }
    for (;;) {
        int g = -1;
#pragma unroll
        for (int i = 0; i < FM; ++i)
            if (g < 0 && left[i])
                g = __builtin_amdgcn_readlane(id[i], __builtin_ctz(left[i]));
        if (g < 0)
            return;
#pragma unroll
        for (int i = 0; i < FM; ++i)
            left[i] &= ~(unsigned)__ballot(id[i] == g);
        const float s = a.scale[g];
        for (int r0 = 0; r0 < a.r; r0 += 16) {
            const int i0 = r0 + half * 8;
            u32v4_t h[FM][3];
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                float v[8] = {};
                if (id[i] == g)
                    adapter_h8(a, M, m0 + i * 32 + l32, i0, s, v);
                split8(v, h[i]);
            }
            auto columns = [&](auto type) {
                typedef decltype(type) T;
                const typename T::raw *up = (const typename T::raw *)a.up + ((long long)g * a.r + i0) * N;
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    const int n = n0 + j * 32 + l32;
                    float u[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        u[e] = n < N && i0 + e < a.r ? load1<T>(up + (long long)e * N + n) : 0.f;
                    u32v4_t b[split_terms<T>()];
                    split8(u, b);
#pragma unroll
                    for (int i = 0; i < FM; ++i) {
                        const f32x16_t t = mfma_terms32(b, h[i], acc[i][j]);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            acc[i][j][e] = id[i] == g ? t[e] : acc[i][j][e];
                    }
                }
            };
            if (a.dtype == CONVIMG_BF16)
                columns(Bf16{});
            else if (a.dtype == CONVIMG_FP16)
                columns(Fp16{});
            else
                columns(Fp32{});
        }
    }
}

}  // namespace convimg
