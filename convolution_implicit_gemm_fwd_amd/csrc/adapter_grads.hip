// adapter_grads.hip -- gradients of the adapters: for each adapter g
//
//   out[i][c] = scale_g * sum over the rows m with ids[m] = g of u[m][i] * v[m][c]
//
// (u = t, v = x for down; u = h, v = dy for up).  The contracted axis is the
// rows, of which an adapter has any number at any places.
#include "adapter.hpp"

namespace convimg {

struct Kept {      // rows kept in 8 bits
    typedef unsigned char raw;
};

// Eight values of a row of v.
template <typename V>
struct Grad8 {
    Raw8<V> r;

    __device__ __forceinline__ void load(const AdGradArgs &a, int m, int c)
    {
        r = tail8<V>(load_raw8<V>((const typename V::raw *)a.v + m * a.ldv, c, a.C), c, a.C);
    }
    __device__ __forceinline__ float get(int e) const
    {
        if constexpr (V::code == CONVIMG_FP32) {
            return __uint_as_float(r.w[e / 4][e % 4]);
        } else {
            const unsigned w = r.w[0][e / 2];
            if constexpr (V::code == CONVIMG_BF16)
                return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
            else
                return (float)__builtin_bit_cast(f16x2_t, w)[e & 1];
        }
    }
};
template <>
struct Grad8<Kept> {
    uint2 q;
    float unit;

    __device__ __forceinline__ void load(const AdGradArgs &a, int m, int c)
    {
        q = uint2{0, 0};
        unit = 0.f;
        if (c < a.C) {
            q = *(const uint2 *)((const unsigned char *)a.v + (long long)m * ((a.C + 31) & ~31) + c);
            unit = mxi_unit(a.vs, m, a.C, c);
        }
    }
    __device__ __forceinline__ float get(int e) const
    {
        return (float)(signed char)((e < 4 ? q.x : q.y) >> (8 * (e & 3))) * unit;
    }
};

template <typename V>
constexpr int grad_terms()
{
    if constexpr (__is_same(V, Kept))
        return 1;
    else
        return split_terms<V>();
}

// A workgroup takes 128 columns, 16 RT ranks of one adapter and one part of
// the rows.  Each of its four waves walks the part's ids and lists the
// adapter's rows, of which it takes every fourth run of 32: lane l loads eight
// columns (l % 16) of eight rows (l / 16) and turns them over in registers to
// the matrix instruction's operand, eight consecutive rows of one column.
// Rows of other adapters are not loaded.
constexpr int kAdGradCols = 128, kAdGradWaves = 4, kAdGradRows = 2048;      // rows listed at once

template <typename V, int RT>
__global__ __launch_bounds__(kAdGradWaves * 64) void ad_grad(AdGradArgs a, int splits, int tiles, int chunks,
                                                             long long first, long long end)
{
    __shared__ __attribute__((aligned(16))) int list[kAdGradWaves][kAdGradRows / kAdGradWaves + 32];
    __shared__ f32x4_t sums[kAdGradWaves - 1][8][64];
    constexpr int NV = grad_terms<V>();
    long long b = first + blockIdx.x;
    if (b >= end)
        return;
    const int tile = (int)(b % tiles);
    b /= tiles;
    const int chunk = (int)(b % chunks);
    b /= chunks;
    const int g = (int)(b % a.G), split = (int)(b / a.G);
    const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = tile * kAdGradCols + r16 * 8, i0 = chunk * 16 * RT;
    const int per = (int)((a.M + (long long)splits - 1) / splits), lo = min((long long)a.M, (long long)split * per),
              hi = min((long long)a.M, (long long)lo + per);
    int *mine = list[wave];
    f32x4_t acc[RT][8] = {};
    int total = 0;

    for (int s0 = lo; s0 < hi; s0 += kAdGradRows) {
        const int s1 = min(hi, s0 + kAdGradRows);
        int n = 0;      // the adapter's rows so far
        for (int m = s0; m < s1; m += 64) {
            const bool is = m + lane < s1 && a.ids[m + lane] == g;
            const unsigned long long all = __ballot(is);
            if (is) {
                const int p = n + __builtin_amdgcn_mbcnt_hi((unsigned)(all >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)all, 0));
                if (((p >> 5) & (kAdGradWaves - 1)) == wave)
                    mine[(p >> 7) * 32 + (p & 31)] = m + lane;
            }
            n += __builtin_popcountll(all);
        }
        total += n;
        mx_wait_lds();      // (the list is the wave's own)
        __builtin_amdgcn_wave_barrier();
        for (int run = wave; run * 32 < n; run += kAdGradWaves) {
            const int slot = (run >> 2) * 32 + q * 8, have = n - run * 32 - q * 8;      // of the lane's eight
            int row[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                row[e] = e < have ? mine[slot + e] : -1;
            Grad8<V> v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = {};
                if (row[e] >= 0)
                    v[e].load(a, row[e], c);
            }
            u32v4_t uf[RT][3];
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const int i = i0 + t * 16 + r16;
                float u[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    u[e] = row[e] >= 0 && i < a.r ? a.u[(long long)row[e] * a.r + i] : 0.f;
                split8(u, uf[t]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    w[e] = v[e].get(j);
                u32v4_t vf[NV];
                split8(w, vf);
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    acc[t][j] = mfma_terms16(uf[t], vf, acc[t][j]);
            }
        }
        __builtin_amdgcn_wave_barrier();
    }

    // the waves' sums in order; a lane holds ranks 4 q .. 4 q + 3 of its eight columns
    if (splits > 1) {
        if (tile == 0 && chunk == 0 && threadIdx.x == 0)
            a.count[(long long)split * a.G + g] = total;
        if (total == 0)
            return;
    }
    const float s = a.scale[g];
    float *out = (splits > 1 ? a.part + (long long)split * a.G * a.r * a.C : a.out) + (long long)g * a.r * a.C;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        __syncthreads();
        if (wave > 0)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                sums[wave - 1][j][lane] = acc[t][j];
        __syncthreads();
        if (wave > 0)
            continue;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int w = 0; w < kAdGradWaves - 1; ++w)
                acc[t][j] += sums[w][j][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = i0 + t * 16 + q * 4 + e;
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                o[j] = total > 0 ? acc[t][j][e] * s : 0.f;
            if (i < a.r && c < a.C)
                store8<Fp32>(out + (long long)i * a.C, c, a.C, o);
        }
    }
}

// The parts' sums in order, without the parts in which the adapter has no rows.
__global__ __launch_bounds__(256) void ad_grad_sum(AdGradArgs a, int splits)
{
    const long long per = (long long)a.r * a.C, all = per * a.G;
    for (long long p = (long long)blockIdx.x * 256 + threadIdx.x; p < all; p += (long long)gridDim.x * 256) {
        const int g = (int)(p / per);
        float s = 0.f;
        for (int k = 0; k < splits; ++k)
            if (a.count[(long long)k * a.G + g] > 0)
                s += a.part[k * all + p];
        a.out[p] = s;
    }
}

int grad_ranks(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : 4; }

int adapter_grad_splits(int M, int C, int G, int r)
{
    const long long rt = 16 * grad_ranks(r), blocks = (C + kAdGradCols - 1LL) / kAdGradCols * G * ((r + rt - 1) / rt);
    const long long want = (2047 + blocks) / blocks, most = (M + 511LL) / 512;
    const long long n = want < most ? want : most;
    return n < 1 ? 1 : n > 64 ? 64 : (int)n;
}

void adapter_grad(const AdGradArgs &a, int v_dtype, int splits, hipStream_t stream)
{
    auto launch = [&](auto v, auto rt) {
        constexpr int RT = decltype(rt)::value;
        const int tiles = (int)((a.C + kAdGradCols - 1LL) / kAdGradCols), chunks = (a.r + 16 * RT - 1) / (16 * RT);
        const long long blocks = (long long)tiles * chunks * a.G * splits;
        constexpr long long kStep = 1 << 22;      // (a launch holds fewer than 2^32 threads)
        for (long long first = 0; first < blocks; first += kStep) {
            const long long n = blocks - first < kStep ? blocks - first : kStep;
            hipLaunchKernelGGL((ad_grad<decltype(v), RT>), dim3((unsigned)n), dim3(kAdGradWaves * 64), 0, stream, a, splits,
                               tiles, chunks, first, blocks);
        }
    };
    auto ranks = [&](auto v) {
        switch (grad_ranks(a.r)) {
        case 1: launch(v, std::integral_constant<int, 1>{}); break;
        case 2: launch(v, std::integral_constant<int, 2>{}); break;
        default: launch(v, std::integral_constant<int, 4>{}); break;
        }
    };
    if (v_dtype == CONVIMG_MXINT8)
        ranks(Kept{});
    else
        with_dtype(v_dtype, ranks);
    if (splits > 1) {
        const long long n = ((long long)a.G * a.r * a.C + 255) / 256;
        hipLaunchKernelGGL(ad_grad_sum, dim3((unsigned)(n < (1 << 20) ? n : (1 << 20))), dim3(256), 0, stream, a, splits);
    }
}

}  // namespace convimg
