// adapter_grads.hpp -- gradients of the adapters: for each adapter g
//
//   out[i][c] = scale_g * sum over the rows m with ids[m] = g of u[m][i] * v[m][c]
//
// (u = t, v = x for down; u = h, v = dy for up).  The contracted axis is the
// rows, of which an adapter has any number at any places.
#pragma once

#include "adapter.hpp"

namespace convimg {

struct Kept {      // rows kept in 8 bits
    typedef unsigned char raw;
};

// Eight columns of eight rows of v, a row an element, and the matrix
// instruction's operand from them: one column of the eight rows, as terms.
template <typename V>
struct Grad8x8 {
    static constexpr int TERMS = split_terms<V>();
    Raw8<V> r[8];

    __device__ __forceinline__ void load(const AdGradArgs &a, int e, int m, int c)
    {
        r[e] = tail8<V>(load_raw8<V>((const typename V::raw *)a.v + m * a.ldv, c, a.C), c, a.C);
    }
    __device__ __forceinline__ void clear(int e) { r[e] = {}; }
    static __device__ __forceinline__ float value(const AdGradArgs &a, int m, int c)
    {
        return load1<V>((const typename V::raw *)a.v + m * a.ldv + c);
    }
    __device__ __forceinline__ void column(int j, u32v4_t (&t)[TERMS]) const
    {
        if constexpr (V::code == CONVIMG_BF16) {      // (the halves of the rows' words, two and two)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                t[0][e] = __builtin_amdgcn_perm(r[2 * e + 1].w[0][j / 2], r[2 * e].w[0][j / 2],
                                                j & 1 ? 0x07060302u : 0x05040100u);
        } else {
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (V::code == CONVIMG_FP32) {
                    w[e] = __uint_as_float(r[e].w[j / 4][j % 4]);
                } else {      // (the word by value: a bit cast of a vector's element takes the first)
                    const unsigned two = r[e].w[0][j / 2];
                    w[e] = (float)__builtin_bit_cast(f16x2_t, two)[j & 1];
                }
            }
            split8(w, t);
        }
    }
};
template <>
struct Grad8x8<Kept> {
    static constexpr int TERMS = 1;
    uint2 q[8];
    float unit[8];

    __device__ __forceinline__ void load(const AdGradArgs &a, int e, int m, int c)
    {
        q[e] = uint2{0, 0};
        unit[e] = 0.f;
        if (c < a.C) {
            q[e] = *(const uint2 *)((const unsigned char *)a.v + (long long)m * ((a.C + 31) & ~31) + c);
            unit[e] = mxi_unit(a.vs, m, a.C, c);
        }
    }
    __device__ __forceinline__ void clear(int e)
    {
        q[e] = uint2{0, 0};
        unit[e] = 0.f;
    }
    static __device__ __forceinline__ float value(const AdGradArgs &a, int m, int c)
    {
        return (float)((const signed char *)a.v)[(long long)m * ((a.C + 31) & ~31) + c] * mxi_unit(a.vs, m, a.C, c);
    }
    __device__ __forceinline__ void column(int j, u32v4_t (&t)[1]) const
    {
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e] = (float)(signed char)((j < 4 ? q[e].x : q[e].y) >> (8 * (j & 3))) * unit[e];
        split8(w, t);
    }
};

// A workgroup takes 128 columns, 16 RT ranks and one chunk of the sorted rows,
// adapter by adapter; of an adapter's rows each of the four waves takes every
// fourth run of 32: lane l loads eight columns (l % 16) of eight rows (l / 16)
// and turns them over in registers to the matrix instruction's operand, eight
// consecutive rows of one column.
//
// An adapter whose rows lie in one chunk is finished there; one that goes on
// leaves its sum in the chunk's first slot if it begins with the chunk, else in
// the second.
//
// 8192 rows of 4 adapters, 16 ranks, 4096 columns of dy (bf16) and 4096 of x (8
// bits): 32.3 us for both gradients, 118 MB read (3.7 TB/s), 7.1 for the sums
// over the chunks; 32 ranks 48.7 and 9, 64 ranks 109 and 15.  Each run of 32 rows
// waits for its order, then for its rows; the waves of other workgroups are what
// covers that, three a SIMD with 16- or 8-bit rows and 16 ranks, one with fp32 rows
// or 32 ranks, none above.
constexpr int kAdGradCols = 128, kAdGradWaves = 4;

template <typename V, int RT>
__device__ __forceinline__ void ad_grad_body(const AdGradArgs &a, unsigned b, f32x4_t (*sums)[8][64])
{
    const int tile = (int)(b % (unsigned)a.tiles);
    b /= (unsigned)a.tiles;
    const int i0 = (int)(b % (unsigned)a.ranks) * 16 * RT, chunk = (int)(b / (unsigned)a.ranks);
    const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = tile * kAdGradCols + r16 * 8;
    const int lo = chunk * a.per, hi = min(a.start[a.G], lo + a.per);

    for (int s0 = lo, s1; s0 < hi; s0 = s1) {
        const int g = a.key[s0], g0 = a.start[g], g1 = a.start[g + 1];
        s1 = min(hi, g1);
        f32x4_t acc[RT][8] = {};
        // (one run after another: two at once take the registers of half the
        // waves, 46 us against 34 for 8192 x (4096 + 4096))
        for (int p0 = s0 + wave * 32; p0 < s1; p0 += kAdGradWaves * 32) {
            // the lane's eight places and rows, in the last run as far as there are any
            const int at = p0 + q * 8;
            const bool whole = p0 + 32 <= s1;
            int row[8];
            if (whole) {
                __builtin_memcpy(row, a.order + at, sizeof(row));
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    row[e] = a.order[min(at + e, s1 - 1)];
            }
            Grad8x8<V> v;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v.load(a, e, row[e], c);
            float u[RT][8];
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const int i = min(i0 + t * 16 + r16, a.r - 1);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    u[t][e] = a.u[(long long)(a.u_sorted ? min(at + e, s1 - 1) : row[e]) * a.u_ld + i];
            }
            if (!whole)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (at + e >= s1) {
                        v.clear(e);
#pragma unroll
                        for (int t = 0; t < RT; ++t)
                            u[t][e] = 0.f;
                    }
            u32v4_t uf[RT][3];
#pragma unroll
            for (int t = 0; t < RT; ++t)
                split8(u[t], uf[t]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                u32v4_t vf[Grad8x8<V>::TERMS];
                v.column(j, vf);
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    acc[t][j] = mfma_terms16(uf[t], vf, acc[t][j]);
            }
        }
        // the waves' sums in order; a lane holds ranks 4 q .. 4 q + 3 of its eight columns
        const bool whole = s0 == g0 && s1 == g1, several = s1 - s0 > 32;
        const float s = a.scale[g];
        float *out = whole ? a.out + (long long)g * a.r * a.C
                           : a.part + ((long long)chunk * 2 + (s0 == lo ? 0 : 1)) * a.r * a.C;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            if (several) {
                __syncthreads();
                if (wave > 0)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        sums[wave - 1][j][lane] = acc[t][j];
                __syncthreads();
            }
            if (wave > 0)
                continue;
            if (several)
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int w = 0; w < kAdGradWaves - 1; ++w)
                        acc[t][j] += sums[w][j][lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = i0 + t * 16 + q * 4 + e;
                float o[8];
                bool nan = false;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    o[j] = acc[t][j][e] * s;
                    nan |= o[j] != o[j];
                }
                if (i < a.r && c < a.C)
                    store8<Fp32>(out + (long long)i * a.C, c, a.C, o);
                if (nan)
                    *a.nan = 1;
            }
        }
    }
}

// Both operands' gradients in one launch, up's first.  16 ranks of 16- and 8-bit
// rows: four waves a SIMD, for which the compiler would take two registers too many.
template <typename DY, typename X, int RT>
__global__ __launch_bounds__(kAdGradWaves * 64, RT == 1 && !__is_same(DY, Fp32) && !__is_same(X, Fp32) ? 4 : 1)
void ad_grad(AdGradArgs up, AdGradArgs down, unsigned up_blocks)
{
    __shared__ f32x4_t sums[kAdGradWaves - 1][8][64];
    if (blockIdx.x < up_blocks)
        ad_grad_body<DY, RT>(up, blockIdx.x, sums);
    else
        ad_grad_body<X, RT>(down, blockIdx.x - up_blocks, sums);
}

// One value of a gradient, value by value.
template <typename V>
__device__ __forceinline__ float ad_grad_value(const AdGradArgs &a, int g, int i, int c)
{
    float s = 0.f;
#pragma unroll 4
    for (int p = a.start[g]; p < a.start[g + 1]; ++p) {
        const int m = a.order[p];
        s = __builtin_fmaf(a.u[(long long)(a.u_sorted ? p : m) * a.u_ld + i], Grad8x8<V>::value(a, m, c), s);
    }
    return s * a.scale[g];
}

// The sums of the adapters whose rows lie in several chunks, in order, and
// zeros for those without rows.  An infinity of one operand times a lower term of
// the other, which may be 0, makes NaN: where some sum is NaN, those are taken
// once more.  (Here, where registers are free: in ad_grad they cost a wave a SIMD.)
template <typename DY, typename X>
__global__ __launch_bounds__(256) void ad_grad_sum(AdGradArgs up, AdGradArgs down)
{
    const AdGradArgs &a = blockIdx.z == 0 ? up : down;
    const long long per = (long long)a.r * a.C;
    const int nan = *a.nan;
    for (int g = blockIdx.y; g < a.G; g += gridDim.y) {
        const int g0 = a.start[g], g1 = a.start[g + 1];
        const int first = g0 / a.per, last = (g1 - 1) / a.per;
        if (g0 < g1 && first == last)
            continue;
        for (long long p = (long long)blockIdx.x * 256 + threadIdx.x; p < per; p += (long long)gridDim.x * 256) {
            float s = 0.f;
            if (g0 < g1) {
                s = a.part[(first * 2LL + (g0 == first * a.per ? 0 : 1)) * per + p];
#pragma unroll 8
                for (int k = first + 1; k <= last; ++k)
                    s += a.part[k * 2LL * per + p];
            }
            a.out[g * per + p] = s;
        }
    }
    if (!nan)
        return;
    for (int g = blockIdx.y; g < a.G; g += gridDim.y)
        for (long long p = (long long)blockIdx.x * 256 + threadIdx.x; p < per; p += (long long)gridDim.x * 256) {
            float &out = a.out[g * per + p];
            const int i = (int)(p / a.C), c = (int)(p - (long long)i * a.C);
            if (out != out)
                out = blockIdx.z == 0 ? ad_grad_value<DY>(a, g, i, c) : ad_grad_value<X>(a, g, i, c);
        }
}

// 16 RT ranks a workgroup, which reads v for all of them: the largest RT that the
// ranks fill.  The registers that more ranks take cost waves, four a SIMD at RT 1,
// two at 2 and one at 4 (fp32 two, two, one), and that is more than they save: 8192
// rows of 4 adapters with x kept, 4096 + 4096 columns, the whole call without dx,
// with RT 1, 2 and 4: 16 ranks 72, 85 and 142 us, 32 ranks 88, 93 and 146, 64 ranks
// 129, 127 and 165, 128 ranks 222, 208 and 250; 2048 rows of 8, 64 ranks: 65, 75 and
// 103.
inline int grad_ranks(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : 4; }

// The launches for one type of dy.
template <typename DY>
void adapter_grads_of(const AdGradArgs &up, const AdGradArgs &down, int x_dtype, hipStream_t stream)
{
    const unsigned n_up = (unsigned)up.tiles * up.ranks * up.chunks, n_down = (unsigned)down.tiles * down.ranks * down.chunks;
    const long long n = ((long long)up.r * (up.C > down.C ? up.C : down.C) + 255) / 256;
    auto launch = [&](auto x, auto rt) {
        hipLaunchKernelGGL((ad_grad<DY, decltype(x), decltype(rt)::value>), dim3(n_up + n_down), dim3(kAdGradWaves * 64), 0,
                           stream, up, down, n_up);
    };
    auto ranks = [&](auto x) {
        switch (grad_ranks(up.r)) {
        case 1: launch(x, std::integral_constant<int, 1>{}); break;
        case 2: launch(x, std::integral_constant<int, 2>{}); break;
        default: launch(x, std::integral_constant<int, 4>{}); break;
        }
        hipLaunchKernelGGL((ad_grad_sum<DY, decltype(x)>),
                           dim3((unsigned)(n < 256 ? n : 256), (unsigned)(up.G < 4096 ? up.G : 4096), 2), dim3(256), 0,
                           stream, up, down);
    };
    if (x_dtype == CONVIMG_MXINT8)
        ranks(Kept{});
    else
        with_dtype(x_dtype, ranks);
}

}  // namespace convimg
