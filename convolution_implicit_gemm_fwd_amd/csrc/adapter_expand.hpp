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
    const void *up;        // [G][r][N]
    const float *scale;    // [G]
    const int *ids;        // [rows]
    const int *order;      // [M]: the row at each place of h and of the product, or NULL for their own order
    int G, r, splits, dtype;

    __device__ __forceinline__ int row(int m) const { return order ? order[m] : m; }
};

// The same with up's type known when compiled.
template <typename T>
struct MxAdapters : MxAdapterArgs {
    typedef T type;
};

// Eight ranks of a row from i0 on, the parts' sums, zeros past the rank.
// (Loads are unconditional, at clamped places: a branch around each would make
// the wave wait for them one by one.)
__device__ __forceinline__ void adapter_h8(const MxAdapterArgs &a, int M, int m, int i0, float (&v)[8])
{
    const float *p = a.h + (long long)m * a.r;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = 0.f;
    for (int k = 0; k < a.splits; ++k, p += (long long)M * a.r) {
        float u[8];
        if (a.r >= 8) {
            unpack8<Fp32>(load_raw8<Fp32, false>(p, i0, a.r), u);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                u[e] = p[min(i0 + e, a.r - 1)];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] += u[e];
    }
    if (a.r >= 8) {
        Raw8<Fp32> w;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w.w[e / 4][e % 4] = __float_as_uint(v[e]);
        unpack8<Fp32>(tail8<Fp32, false>(w, i0, a.r), v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = i0 + e < a.r ? v[e] : 0.f;
    }
}

// Adds to the sums of FM x FN blocks of 32 x 32 from row m0 and column n0 on; a
// lane holds row lane % 32 of a block and 16 of its columns (the instruction's
// rows).
//
// For 16 ranks at a time the wave goes through the adapters that its rows have,
// in the order of their first rows, P of them in flight at once; of KG groups
// of waves that share the tile each takes every KG-th.  A row has zeros for h
// in another adapter's product.  Zero times an infinity would not do: such
// values of up are left out (0) here, and the answer says that there are some,
// for adapter_infinite.  (Selecting by row after the product instead takes the
// sums from the matrix unit's registers: the largest tile then spills.)
template <typename T, int FM, int FN, int KG>
__device__ __forceinline__ bool adapter_expand(const MxAdapterArgs &a, int M, int N, int m0, int n0, int group,
                                               f32x16_t (&acc)[FM][FN])
{
    constexpr int P = FM * FN <= 1 ? 8 : FM * FN <= 2 ? 4 : FM * FN <= 4 ? 2 : 1;
    const int lane = threadIdx.x & 63, half = lane >> 5, l32 = lane & 31;
    int id[FM];
    float s[FM];
    unsigned any[FM];
    bool infinite = false;
#pragma unroll
    for (int i = 0; i < FM; ++i)
        id[i] = a.ids[a.row(min(m0 + i * 32 + l32, M - 1))];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        id[i] = m0 + i * 32 + l32 < M && id[i] < a.G ? id[i] : -1;
        s[i] = a.scale[max(id[i], 0)];
        any[i] = (unsigned)__ballot(id[i] >= 0);
    }
    // (one pass through each loop at least, without a branch around: the sums stay where they are)
    int r0 = 0, turn = group;
    do {
        const int i0 = r0 + half * 8;
        u32v4_t h[FM][3];
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            float v[8];
            adapter_h8(a, M, min(m0 + i * 32 + l32, M - 1), i0, v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] *= s[i];
            split8(v, h[i]);
        }
        unsigned left[FM], rest;
#pragma unroll
        for (int i = 0; i < FM; ++i)
            left[i] = any[i];
        int number = 0;      // of the adapter among the tile's
        do {
            int g[P];
            typename T::raw w[P][FN][8];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                for (;;) {
                    g[p] = -2;
#pragma unroll
                    for (int i = 0; i < FM; ++i)
                        if (g[p] < 0 && left[i])
                            g[p] = __builtin_amdgcn_readlane(id[i], __builtin_ctz(left[i]));
#pragma unroll
                    for (int i = 0; i < FM; ++i)
                        left[i] &= ~(unsigned)__ballot(id[i] == g[p]);
                    if (KG == 1 || g[p] < 0 || (number++ + turn) % KG == 0)
                        break;
                }
                const typename T::raw *up = (const typename T::raw *)a.up + (long long)max(g[p], 0) * a.r * N;
#pragma unroll
                for (int j = 0; j < FN; ++j)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        w[p][j][e] = up[(long long)min(i0 + e, a.r - 1) * N + min(n0 + j * 32 + l32, N - 1)];
            }
#pragma unroll
            for (int p = 0; p < P; ++p) {
                u32v4_t hm[FM][3];
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int k = 0; k < 3; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            hm[i][k][e] = id[i] == g[p] ? h[i][k][e] : 0u;
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    float u[8];
                    bool odd = false;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        u[e] = i0 + e < a.r ? load1<T>(&w[p][j][e]) : 0.f;
                        const bool fine = __builtin_fabsf(u[e]) < __builtin_inff();
                        odd |= !fine;
                        u[e] = fine ? u[e] : 0.f;
                    }
                    infinite |= __any(odd);
                    u32v4_t b[split_terms<T>()];
                    split8(u, b);
#pragma unroll
                    for (int i = 0; i < FM; ++i)
                        acc[i][j] = mfma_terms32(b, hm[i], acc[i][j]);
                }
            }
            rest = 0;
#pragma unroll
            for (int i = 0; i < FM; ++i)
                rest |= left[i];
        } while (rest);
        r0 += 16;
        ++turn;
    } while (r0 < a.r);
    return infinite;
}

// The outputs that an infinity or a NaN in up reaches, over what was stored for
// them: TM x TN of them from row m0 and column n0 on, by one wave.
template <typename T, typename O>
__device__ __forceinline__ void adapter_infinite(const MxAdapterArgs &a, int M, int N, int m0, int n0, int TM, int TN,
                                                 void *out)
{
    for (int k = threadIdx.x & 63; k < TM * TN; k += 64) {
        const int m = m0 + k / TN, n = n0 + k % TN, row = a.row(min(m, M - 1)), id = m < M && n < N ? a.ids[row] : -1;
        if (id < 0 || id >= a.G)
            continue;
        float s = 0.f;
        for (int i = 0; i < a.r; ++i) {
            const float u = load1<T>((const typename T::raw *)a.up + ((long long)id * a.r + i) * N + n);
            if (!(__builtin_fabsf(u) < __builtin_inff())) {
                float h = 0.f;
                for (int p = 0; p < a.splits; ++p)
                    h += a.h[((long long)p * M + m) * a.r + i];
                s += h * a.scale[id] * u;
            }
        }
        if (!(__builtin_fabsf(s) < __builtin_inff()))
            store1<O>((typename O::raw *)out + (long long)row * N + n, s);
    }
}

}  // namespace convimg
