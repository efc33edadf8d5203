// adapter_expand.hpp -- the second half of low-rank adapters inside a product:
// adds scale_g h[m] up_g to the sums of a tile whose rows m may belong to
// different adapters g.
//
// Values are split into bf16 terms that add up to them exactly (bf16 1, fp16 2,
// fp32 3 terms of at most 8 bits), so that bf16 matrix instructions give fp32
// products: those of terms i and j with i + j <= 3.  Term i is below 2^(1 - 8 i)
// of the value, so the one product left out, of the last terms of two fp32 values,
// is below 2^-30; without those of i + j = 3, which reach 2^-21 together and all
// have the product's sign, a sum of products would be off by several units in its
// last place.  (The smallest bf16 is 2^-133: an fp32 value's bits below that are
// left out.)
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
    for (int s = 3; s >= 0; --s)
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
    for (int s = 3; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB)
                c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a[i]),
                                                            __builtin_bit_cast(bf16x8_t, b[s - i]), c, 0, 0, 0);
    return c;
}

struct MxNoAdapters {};

// Ranks in whole steps of the matrix instruction.
__host__ __device__ inline int adapter_ranks(int r) { return (r + 15) & ~15; }

// h of a place as the products take it: scaled, for each 16 ranks three terms
// of 16, zeros past the rank.  The terms of an infinity or a NaN are 0, the first
// one with a sign, which no other first term of that size has.
constexpr int kAdTermBytes = 96;

__device__ __forceinline__ void adapter_terms(float h, unsigned short (&t)[3])
{
    const float v[8] = {h};
    u32v4_t s[3];
    split8(v, s);
    const bool finite = __builtin_fabsf(h) < __builtin_inff();
#pragma unroll
    for (int k = 0; k < 3; ++k)
        t[k] = finite ? (unsigned short)s[k][0] : (unsigned short)0;
    t[0] = !finite ? 0x8000 : t[0] == 0x8000 ? 0 : t[0];
}

struct MxAdapterArgs {
    const unsigned char *terms;      // [M][ranks / 16][3][16] bf16, 16-byte aligned
    const float *h;                  // [M][adapter_ranks(r)], not scaled
    const void *up;                  // [G][r][N]
    const float *scale;              // [G]
    const int *key;                  // [M]: the adapter at each place of h and of the product
    const int *order;                // [M]: the output's row at each place, or NULL for their own order
    int G, r, dtype;

    __device__ __forceinline__ int row(int m) const { return order ? order[m] : m; }
};

// The same with up's type known when compiled.
template <typename T>
struct MxAdapters : MxAdapterArgs {
    typedef T type;
};

// Eight loaded values of up as terms; infinities and NaN, of which the answer
// tells, are left out.
template <typename T>
__device__ __forceinline__ bool adapter_up8(const typename T::raw (&w)[8], u32v4_t (&t)[split_terms<T>()])
{
    if constexpr (T::code == CONVIMG_FP32) {
        float u[8];
        unsigned top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top = mx_top(top, u[e] = w[e]);
        const bool odd = __any(top >= 0x7f800000u);
        if (odd)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                u[e] = __builtin_fabsf(u[e]) < __builtin_inff() ? u[e] : 0.f;
        split8(u, t);
        return odd;
    } else {
        typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
        constexpr unsigned short INF = T::code == CONVIMG_BF16 ? 0x7f80 : 0x7c00;
        u16x2 top = {};
        Raw8<T> r;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r.w[0][e] = w[2 * e] | (unsigned)w[2 * e + 1] << 16;
            top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, r.w[0][e] & 0x7fff7fffu));
        }
        const bool odd = __any(max(top[0], top[1]) >= INF);
        if (odd)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const unsigned v = r.w[0][e];
                r.w[0][e] = ((v & 0x7fffu) < INF ? v & 0xffffu : 0u) | ((v >> 16 & 0x7fffu) < INF ? v & 0xffff0000u : 0u);
            }
        split_raw8<T>(r, t);
        return odd;
    }
}

// Adds to the sums of FM x FN blocks of 32 x 32 from place m0 and column n0 on; a
// lane holds place lane % 32 of a block and 16 of its columns (the instruction's
// rows).
//
// The wave goes through the adapters that its places have, in their order, 16
// ranks at a time, P such steps in flight at once (loads are unconditional, at
// clamped places: a branch around each would make the wave wait for them one
// by one); of KG groups of waves that share the tile each takes every KG-th
// step.  A place has zeros for h in another adapter's product.  Zero times an
// infinity would not do, nor an infinity times a value's lower terms, which may be
// 0: values of up that are not finite are left out (0) here, those of h were
// before, and the answer says that there are some of h (1) or of up (2), for
// adapter_infinite.  (Selecting by place after the
// product instead takes the sums from the matrix unit's registers: the largest
// tile then spills, 8192^3 with 16 ranks 777 us.)
//
// The loads' latency bounds it: in the product of 8192^3 it adds nothing that can
// be told from the product's own spread for 4 adapters in runs and 16 ranks (260
// us), 50 us for 64 ranks; in that of 2011 x 4096 x 4096 14 us for 64 ranks; in
// that of 61 x 8000 x 4096 with an adapter a row 6 us, the rows' parts of up
// (8000 x 16 a row) being read from memory then.  (Three steps in flight instead of
// two in the 128 x 128 tiles, for which there are registers: 2011 x 4096 x 4096 with
// 64 ranks, the whole call, 60.1 us against 59.5.)
template <typename T, int FM, int FN, int KG>
__device__ __forceinline__ unsigned adapter_expand(const MxAdapterArgs &a, int M, int N, int m0, int n0, int group,
                                               f32x16_t (&acc)[FM][FN])
{
    constexpr int P = FM * FN <= 1 ? 8 : FM * FN <= 2 ? 4 : 2, NT = split_terms<T>();
    const int lane = threadIdx.x & 63, half = lane >> 5, l32 = lane & 31;
    const int steps = adapter_ranks(a.r) / 16;
    int id[FM];
    unsigned any[FM], left[FM];
    typedef short i16x2 __attribute__((ext_vector_type(2)));
    i16x2 low = {};
    bool infinite = false;
#pragma unroll
    for (int i = 0; i < FM; ++i)
        id[i] = a.key[min(m0 + i * 32 + l32, M - 1)];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        id[i] = m0 + i * 32 + l32 < M && id[i] < a.G ? id[i] : -1;
        left[i] = any[i] = (unsigned)__ballot(id[i] >= 0);
    }
    int step = 0, number = 0;
    // the next adapter, -2 for none, and (in step) its 16 ranks
    auto next = [&]() {
        for (;;) {
            int g = -2;
#pragma unroll
            for (int i = 0; i < FM; ++i)
                if (g < 0 && left[i])
                    g = __builtin_amdgcn_readlane(id[i], __builtin_ctz(left[i]));
            if (g < 0) {
                unsigned some = 0;
#pragma unroll
                for (int i = 0; i < FM; ++i)
                    some |= left[i] = any[i];
                if (!some || step + 1 >= steps) {
#pragma unroll
                    for (int i = 0; i < FM; ++i)
                        left[i] = any[i] = 0;
                    return g;
                }
                ++step;
                continue;
            }
#pragma unroll
            for (int i = 0; i < FM; ++i)
                left[i] &= ~(unsigned)__ballot(id[i] == g);
            if (KG == 1 || number++ % KG == group)
                return g;
        }
    };
    int g0 = next();
    if (g0 < 0)
        return 0;
    do {
        int g[P];
        u32v4_t h[P][FM][3];
        typename T::raw w[P][FN][8];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            g[p] = p == 0 ? g0 : next();
            if (g[p] < 0)
                continue;
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const u32v4_t *from = (const u32v4_t *)(a.terms + ((long long)min(m0 + i * 32 + l32, M - 1) * steps + step)
                                                                     * kAdTermBytes) + half;
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    h[p][i][k] = from[2 * k];
            }
            const typename T::raw *up = (const typename T::raw *)a.up + (long long)g[p] * a.r * N;
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    w[p][j][e] = up[(long long)min(step * 16 + half * 8 + e, a.r - 1) * N + min(n0 + j * 32 + l32, N - 1)];
        }
        g0 = g[P - 1] < 0 ? -2 : next();
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if (g[p] < 0)
                continue;
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int k = 0; k < 3; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const unsigned v = id[i] == g[p] ? h[p][i][k][e] : 0u;
                        h[p][i][k][e] = v;
                        if (k == 0)
                            low = __builtin_elementwise_min(low, __builtin_bit_cast(i16x2, v));
                    }
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                u32v4_t b[NT];
                infinite |= adapter_up8<T>(w[p][j], b);
#pragma unroll
                for (int i = 0; i < FM; ++i)
                    acc[i][j] = mfma_terms32(b, h[p][i], acc[i][j]);
            }
        }
    } while (g0 >= 0);
    return (__any(min(low[0], low[1]) == -32768) ? 1u : 0u) | (infinite ? 2u : 0u);
}

// Adds what was left out of h and of up, as far as `left` says there is, to the
// outputs that it reaches, of which the rest was stored: TM x TN of them from row
// m0 and column n0 on, by one wave.  (An infinity that the rest is in fp16, but
// not the bias, counts as a sum past fp16's largest value, which is finite before
// it is rounded; where scale h is past fp32's largest value and the sum is not, the
// output is rounded twice.)
template <typename T, typename O>
__device__ __forceinline__ void adapter_infinite(const MxAdapterArgs &a, const float *bias, int M, int N, int m0, int n0,
                                                 int TM, int TN, unsigned left, void *out)
{
    auto finite = [](float v) { return __builtin_fabsf(v) < __builtin_inff(); };
    const int lane = threadIdx.x & 63;
    for (int base = m0; base < min(m0 + TM, M); base += 64) {
        // a lane a row: its adapter, and whether something of its h was left out
        const int mine = min(base + lane, M - 1), given = base + lane < min(m0 + TM, M) ? a.key[mine] : -1;
        bool some = (left & 2) != 0;
        if (given >= 0 && given < a.G)
            for (int i = 0; i < a.r; ++i)
                some |= !finite(a.h[(long long)mine * adapter_ranks(a.r) + i] * a.scale[given]);
        for (unsigned long long rows = __ballot(some && given >= 0 && given < a.G); rows; rows &= rows - 1) {
            const int k = __builtin_ctzll(rows), m = base + k, id = __builtin_amdgcn_readlane(given, k);
            const float *h = a.h + (long long)m * adapter_ranks(a.r), scale = a.scale[id];
            const typename T::raw *up = (const typename T::raw *)a.up + (long long)id * a.r * N;
            for (int n = n0 + lane; n < min(n0 + TN, N); n += 64) {
                typename O::raw *o = (typename O::raw *)out + (long long)a.row(m) * N + n;
                float rest = load1<O>(o), s = 0.f;
                if (rest != rest)
                    continue;
                bool any = false;
                for (int i = 0; i < a.r; ++i) {
                    const float u = load1<T>(up + (long long)i * N + n);
                    if (!finite(u) || !finite(h[i] * scale)) {
                        s = __builtin_fmaf(h[i], u, s);
                        any = true;
                    }
                }
                if (!any)
                    continue;
                s *= scale;
                if (O::code == CONVIMG_FP16 && __builtin_isinf(rest) && !(bias && __builtin_isinf(bias[n])) && !finite(s))
                    rest = 0.f;
                store1<O>(o, rest + s);
            }
        }
    }
}

}  // namespace convimg
