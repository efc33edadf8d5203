// adapter_shrink.hip -- h[m] = down_g x[m], g = ids[m], in one pass over x
// that also writes x's MXFP4 rows for the shared projection and, for training,
// its MXINT8 rows.
#include "adapter.hpp"

namespace convimg {

// ---- few rows --------------------------------------------------------------
//
// A workgroup takes kAdFewCols columns of one row, a thread eight of them, with
// its part of every rank's row of the adapter in flight at once: a serving batch
// mostly has another adapter in every row, whose 2 r K bytes are the work.  The
// parts' sums stay apart; what reads h adds them.
constexpr int kAdFewThreads = 128, kAdFewCols = kAdFewThreads * 8, kAdFewRanks = 16;

template <typename X, typename A>
__global__ __launch_bounds__(kAdFewThreads) void ad_shrink_few(AdShrinkArgs a)
{
    __shared__ float sums[2][kAdFewRanks];
    const int m = blockIdx.y, c = blockIdx.x * kAdFewCols + threadIdx.x * 8;
    const int id = a.ids[m];
    const bool has = id >= 0 && id < a.G;
    const Raw8<X> raw = load_raw8<X>((const typename X::raw *)a.x + m * a.ldx, c, a.K);
    float v[8];
    unpack8<X>(tail8<X>(raw, c, a.K), v);
    if (a.codes) {
        unsigned top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top = mx_top(top, v[e]);
        const unsigned byte = mx_scale_byte(quad_max(top));
        const int kb = mx_blocks(a.K);
        if (c < kb * 32)
            ((unsigned *)a.codes)[((long long)m * kb * 32 + c) / 8] = mx_encode8(v, mx_scale_value(byte));
        const unsigned word = mx_scale_word<16>(byte, c >> 5);
        if ((c & 127) == 0 && c < a.K)
            ((unsigned *)a.scales)[(long long)(c >> 7) * a.M + m] = word;
    }
    float *h = a.h + ((long long)blockIdx.x * a.M + m) * a.r;
    const typename A::raw *down = (const typename A::raw *)a.down + (long long)id * a.r * a.K;
    for (int i0 = 0; i0 < a.r; i0 += kAdFewRanks) {
        Raw8<A> w[kAdFewRanks];
        if (has)
#pragma unroll
            for (int i = 0; i < kAdFewRanks; ++i)
                w[i] = load_raw8<A>(down + (long long)min(i0 + i, a.r - 1) * a.K, c, a.K);
        __syncthreads();      // the previous sums have been read
#pragma unroll
        for (int i = 0; i < kAdFewRanks; ++i) {
            float s = 0.f;
            if (has) {
                float u[8];
                unpack8<A>(tail8<A>(w[i], c, a.K), u);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s = __builtin_fmaf(u[e], v[e], s);
            }
            s = group_sum<64>(s);
            if ((threadIdx.x & 63) == 0)
                sums[threadIdx.x >> 6][i] = s;
        }
        __syncthreads();
        if (threadIdx.x < kAdFewRanks && i0 + (int)threadIdx.x < a.r)
            h[i0 + threadIdx.x] = sums[0][threadIdx.x] + sums[1][threadIdx.x];
    }
}

// ---- many rows -------------------------------------------------------------
//
// A workgroup takes 16 rows and 16 RT ranks, its eight waves share the columns
// in steps of 128: a lane holds one block of 32 columns of one row, which it
// quantises by itself, and which is its part of the matrix instructions'
// operand (four steps of 32 columns, eight of each lane; any order of the
// columns will do as long as both operands have it).  The adapters that the 16
// rows have are taken D at a time, each with sums of its own; x is read again
// (from cache) for more.
constexpr int kAdWaves = 8;

// 32 values of a lane: rows of x and of an adapter.
template <typename T>
struct Lane32 {
    Raw8<T> raw[4];

    __device__ __forceinline__ void load(const typename T::raw *row, int c, int cols)
    {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            raw[j] = load_raw8<T>(row, c + 8 * j, cols);
    }
    __device__ __forceinline__ void tail(int c, int cols)
    {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            raw[j] = tail8<T>(raw[j], c + 8 * j, cols);
    }
};

template <typename X, typename A, int RT, int D>
__global__ __launch_bounds__(kAdWaves * 64) void ad_shrink_tile(AdShrinkArgs a)
{
    __shared__ f32x4_t sums[kAdWaves][D * RT][64];
    static_assert(D * RT <= kAdWaves, "a wave a block of sums");
    const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = blockIdx.x * 16, m = m0 + r16, i0 = blockIdx.y * 16 * RT;
    const int kb = mx_blocks(a.K), quads = (a.K + 127) / 128;
    const bool real = m < a.M, write = blockIdx.y == 0;
    const int given = real ? a.ids[m] : -1, id = given < a.G ? given : -1;
    const typename X::raw *x = (const typename X::raw *)a.x + (long long)min(m, a.M - 1) * a.ldx;
    unsigned left = (unsigned)__ballot(id >= 0) & 0xffffu;

    if (real && id < 0)      // no adapter: 0
        for (int i = i0 + (threadIdx.x >> 4); i < min(a.r, i0 + 16 * RT); i += kAdWaves * 4)
            a.h[(long long)m * a.r + i] = 0.f;
    bool first = write;
    do {
        int g[D], n = 0;
#pragma unroll
        for (int d = 0; d < D; ++d) {
            g[d] = -1;
            if (left) {
                g[d] = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
                left &= ~(unsigned)__ballot(id == g[d]);
                n = d + 1;
            }
        }
        f32x4_t acc[D][RT] = {};
        for (int k0 = wave * 128; k0 < quads * 128; k0 += kAdWaves * 128) {
            const int c = k0 + q * 32;
            Lane32<X> xr;
            xr.load(x, c, a.K);
            xr.tail(c, a.K);
            if (first && (a.codes || a.codes8)) {
                float v[32];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float u[8];
                    unpack8<X>(xr.raw[j], u);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[8 * j + e] = u[e];
                }
                const int blk = c >> 5;
                if (a.codes) {
                    u32v4_t code;
                    const unsigned byte = mx_encode32(v, code);
                    if (real && blk < kb)
                        *(u32v4_t *)(a.codes + ((long long)m * kb + blk) * 16) = code;
                    if (real)
                        a.scales[((long long)(k0 >> 7) * a.M + m) * 4 + q] = (unsigned char)(blk < kb ? byte : 0u);
                }
                if (a.codes8) {
                    unsigned top = 0;
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        top = mx_top(top, v[e]);
                    const unsigned byte = mxi_scale_byte(top);
                    uint4 o[2];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float u[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            u[e] = v[8 * j + e];
                        ((uint2 *)o)[j] = mxi_encode8(u, byte);
                    }
                    if (real && blk < kb) {
                        uint4 *p = (uint4 *)(a.codes8 + ((long long)m * kb + blk) * 32);
                        p[0] = o[0];
                        p[1] = o[1];
                    }
                    if (real)
                        a.scales8[(long long)m * (quads * 4) + blk] = (unsigned char)(blk < kb ? byte : 0u);
                }
            }
            if (n == 0)
                continue;
            u32v4_t xf[4][split_terms<X>()];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                split_raw8<X>(xr.raw[j], xf[j]);
#pragma unroll
            for (int d = 0; d < D; ++d)
                if (d < n)
#pragma unroll
                    for (int t = 0; t < RT; ++t) {
                        const int i = min(i0 + t * 16 + r16, a.r - 1);
                        Lane32<A> w;
                        w.load((const typename A::raw *)a.down + ((long long)g[d] * a.r + i) * a.K, c, a.K);
                        w.tail(c, a.K);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            u32v4_t wf[split_terms<A>()];
                            split_raw8<A>(w.raw[j], wf);
                            acc[d][t] = mfma_terms16(wf, xf[j], acc[d][t]);
                        }
                    }
        }
        first = false;
        if (n == 0)
            break;
        // the waves' sums in order; a lane holds ranks 4 q .. 4 q + 3 of row r16
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
            for (int t = 0; t < RT; ++t)
                sums[wave][d * RT + t][lane] = acc[d][t];
        __syncthreads();
        if (wave < D * RT) {
            const int d = wave / RT, t = wave % RT;
            f32x4_t s = sums[0][wave][lane];
#pragma unroll
            for (int w = 1; w < kAdWaves; ++w)
                s += sums[w][wave][lane];
            int mine = -1;
#pragma unroll
            for (int k = 0; k < D; ++k)
                mine = k == d ? g[k] : mine;
            if (mine >= 0 && id == mine)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = i0 + t * 16 + q * 4 + e;
                    if (i < a.r)
                        a.h[(long long)m * a.r + i] = s[e];
                }
        }
        __syncthreads();
    } while (left);
}

// Up to kAdFewM rows go a row a workgroup.
constexpr int kAdFewM = 64;

int adapter_splits(int M, int K, bool whole) { return !whole && M <= kAdFewM ? (K + kAdFewCols - 1) / kAdFewCols : 1; }

void adapter_shrink(const AdShrinkArgs &a, int x_dtype, int a_dtype, int splits, hipStream_t stream)
{
    const bool few = a.M <= kAdFewM && !a.codes8 && splits == (a.K + kAdFewCols - 1) / kAdFewCols;
    with_dtype(x_dtype, [&](auto x) {
        with_dtype(a_dtype, [&](auto w) {
            typedef decltype(x) X;
            typedef decltype(w) A;
            if (few) {
                hipLaunchKernelGGL((ad_shrink_few<X, A>), dim3(splits, a.M), dim3(kAdFewThreads), 0, stream, a);
                return;
            }
            const unsigned tiles = (unsigned)((a.M + 15LL) / 16);
            if (a.r <= 16)
                hipLaunchKernelGGL((ad_shrink_tile<X, A, 1, 4>), dim3(tiles), dim3(kAdWaves * 64), 0, stream, a);
            else if (a.r <= 32)
                hipLaunchKernelGGL((ad_shrink_tile<X, A, 2, 2>), dim3(tiles), dim3(kAdWaves * 64), 0, stream, a);
            else
                hipLaunchKernelGGL((ad_shrink_tile<X, A, 4, 2>), dim3(tiles, (a.r + 63) / 64), dim3(kAdWaves * 64), 0,
                                   stream, a);
        });
    });
}

}  // namespace convimg
