// layer_norm.hpp -- pieces shared by the layer norm kernels: sums over a row's
// threads, the columns of a thread, launch shapes, argument checks and the sums
// over partial parameter gradients.
#pragma once

#include <type_traits>

#include "row_common.hpp"

namespace convimg {

constexpr int kLnThreads = 256;

// Sum over a workgroup of kLnThreads, the same in every thread.
__device__ __forceinline__ float block_sum(float v, float *lds)
{
    v = group_sum<64>(v);
    __syncthreads();   // the previous sum has been read
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// Threads of a workgroup whose rows take TPR threads each.
constexpr int row_threads(int tpr) { return tpr > kLnThreads ? tpr : kLnThreads; }

// Sum of v over the TPR threads of a row, the same in each: part of a wave,
// or the whole workgroup (`lds` then TPR / 64 floats, of alternate buffers in
// consecutive calls, so that one barrier a sum is enough).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *lds)
{
    if constexpr (TPR <= 64) {
        return group_sum<TPR>(v);
    } else {
        v = group_sum<64>(v);
        if ((threadIdx.x & 63) == 0)
            lds[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int w = 0; w < TPR / 64; w += 2)
            v += lds[w] + lds[w + 1];
        return v;
    }
}

// The columns of thread l of a row: V groups of eight, TPR groups apart.  With
// WINDOW the group that the row's end cuts is its last eight columns instead,
// so that loads and stores stay whole; the columns that it shares with its
// neighbour are computed twice, alike, and counted once in the row's sums.
template <int TPR, int V, bool WINDOW>
struct RowCols {
    int col[V];       // first column, at least `cols` for none
    int first[V];     // first of the eight that counts

    __device__ __forceinline__ RowCols(int l, int cols)
    {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * TPR + l) * 8;
            col[i] = WINDOW && c < cols ? min(c, cols - 8) : c;
            first[i] = c < cols ? c - col[i] : 8;
        }
    }
    __device__ __forceinline__ bool counts(int i, int e) const { return e >= first[i]; }

    template <typename T>
    __device__ __forceinline__ Raw8<T> load(const typename T::raw *row, int i, int cols) const
    {
        return load_raw8<T, TPR == 4>(row, col[i], cols);
    }
    template <typename T>
    __device__ __forceinline__ void unpack(const Raw8<T> &r, int i, int cols, float (&v)[8]) const
    {
        unpack8<T>(WINDOW ? r : tail8<T, TPR == 4>(r, col[i], cols), v);
    }
};

__device__ __forceinline__ void store8_as(int dtype, void *p, long long row, int col, int cols, const float (&v)[8])
{
    if (dtype == CONVIMG_FP32)
        store8<Fp32>((float *)p + row * cols, col, cols, v);
    else if (dtype == CONVIMG_BF16)
        store8<Bf16>((unsigned short *)p + row * cols, col, cols, v);
    else
        store8<Fp16>((unsigned short *)p + row * cols, col, cols, v);
}

// Two sums over the TPR threads of a row at once.
template <int TPR>
__device__ __forceinline__ void row_sum2(float &s1, float &s2, float (*lds)[2])
{
    if constexpr (TPR <= 64) {
        s1 = group_sum<TPR>(s1);
        s2 = group_sum<TPR>(s2);
    } else {
        s1 = group_sum<64>(s1);
        s2 = group_sum<64>(s2);
        if ((threadIdx.x & 63) == 0) {
            lds[threadIdx.x >> 6][0] = s1;
            lds[threadIdx.x >> 6][1] = s2;
        }
        __syncthreads();
        s1 = s2 = 0.f;
#pragma unroll
        for (int w = 0; w < TPR / 64; w += 2) {
            s1 += lds[w][0] + lds[w + 1][0];
            s2 += lds[w][1] + lds[w + 1][1];
        }
    }
}

// dgamma and dbeta: the partial sums in a fixed order, 16 columns a workgroup
// and 64 threads a column (512 sums of 128 columns: 3 us; a thread a column took
// 62).  A launch takes the columns from `first`, up to kLnRedStep of the 2
// cols, as it holds fewer than 2^32 threads.
constexpr int kLnRedCols = 16, kLnRedThreads = 1024, kLnRedStep = 1 << 24;

static __global__ __launch_bounds__(kLnRedThreads) void ln_bwd_reduce(const float *part, float *dgamma, float *dbeta,
                                                               int cols, int parts, long long first)
{
    constexpr int LANES = kLnRedThreads / kLnRedCols;
    __shared__ float lds[LANES][kLnRedCols + 1];
    const int k = threadIdx.x % kLnRedCols, p0 = threadIdx.x / kLnRedCols;
    const long long c = first + (long long)blockIdx.x * kLnRedCols + k;
    float s = 0.f;
    if (c < 2LL * cols)
#pragma unroll 4
        for (int p = p0; p < parts; p += LANES)
            s += part[(long long)p * 2 * cols + c];
    lds[p0][k] = s;
    __syncthreads();
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
        if (p0 < o)
            lds[p0][k] += lds[p0 + o][k];
        __syncthreads();
    }
    if (p0 == 0 && c < 2LL * cols) {
        if (c < cols)
            dgamma[c] = lds[0][k];
        else
            dbeta[c - cols] = lds[0][k];
    }
}

inline void ln_reduce_parts(const float *part, float *dgamma, float *dbeta, int cols, int parts, hipStream_t stream)
{
    for (long long c = 0, end = 2LL * cols; c < end; c += kLnRedStep) {
        const long long n = end - c < kLnRedStep ? end - c : kLnRedStep;
        hipLaunchKernelGGL(ln_bwd_reduce, dim3((unsigned)((n + kLnRedCols - 1) / kLnRedCols)), dim3(kLnRedThreads), 0,
                           stream, part, dgamma, dbeta, cols, parts, c);
    }
}

// Rows and columns each fit an int; all element offsets are 64-bit.
inline int ln_check(const void *x, long long ldx, long long rows, int cols, int dtype)
{
    if (rows < 0 || cols <= 0 || ldx < cols)
        return CONVIMG_ERR_SHAPE;
    if (!dtype_ok(dtype))
        return CONVIMG_ERR_DTYPE;
    if (rows > kMaxRows || cols > kMaxCols)
        return CONVIMG_ERR_RANGE;
    if (!x && rows > 0)
        return CONVIMG_ERR_NULL;
    return CONVIMG_OK;
}

// Calls f<TPR, V>() for the threads a row that hold `cols` columns at 8 V
// each: as few threads as one eighth of the columns needs (a power of two, so
// that a wave takes whole rows), up to 1024.  From 513 to 1024 columns a wave
// still holds the row, two groups of eight a thread, and from 1025 a workgroup
// of at least 256 threads does; f<0, 0>() past 8192 columns.
template <typename F>
void with_row_shape(int cols, F &&f)
{
    using std::integral_constant;
    auto call = [&](auto t, auto v) { f(t, v); };
#define CONVIMG_ROWS(T, V) call(integral_constant<int, T>{}, integral_constant<int, V>{})
    if (cols <= 32)
        CONVIMG_ROWS(4, 1);
    else if (cols <= 64)
        CONVIMG_ROWS(8, 1);
    else if (cols <= 128)
        CONVIMG_ROWS(16, 1);
    else if (cols <= 256)
        CONVIMG_ROWS(32, 1);
    else if (cols <= 512)
        CONVIMG_ROWS(64, 1);
    else if (cols <= 1024)
        CONVIMG_ROWS(64, 2);
    else if (cols <= 2048)
        CONVIMG_ROWS(256, 1);
    else if (cols <= 4096)
        CONVIMG_ROWS(512, 1);
    else if (cols <= 8192)
        CONVIMG_ROWS(1024, 1);
    else
        CONVIMG_ROWS(0, 0);
#undef CONVIMG_ROWS
}

// Workgroups for one a row: a launch holds fewer than 2^32 threads, so very
// many rows are walked in strides of the grid.
inline unsigned ln_grid(long long rows) { return (unsigned)(rows < (1 << 22) ? rows : (1 << 22)); }

// Workgroups of the forward pass: at most what 256 CUs hold of 2048 threads,
// which walk the rows.
inline unsigned ln_fwd_grid(long long rows, int tpr, bool eights)
{
    const long long per = row_threads(tpr) / tpr, n = (rows + per - 1) / per;
    const long long most = 256 * 2048 / row_threads(tpr);
    const unsigned g = (unsigned)(n < most ? n : most);
    return eights ? (g + 7) & ~7u : g;
}

// Partial sums of the parameters' gradients, one a workgroup of the
// backward pass: enough workgroups to keep the memory busy, few enough that
// the partial sums (2 cols fp32 each, written and read) stay small beside
// dy, x and dx.  A single one writes the gradients itself: so do up to four
// groups of rows, for which a second launch (4 us) would cost more than the
// other workgroups save.  512 workgroups of 256 threads, 256 of more (65536 x
// 128 16.9 us, 17.8 with 1024; 65536 x 1024 75 us, 88 with 1024; 16384 x 4096
// 79 us, 81 with 512; 8192 x 8192 81 us, 91 with 512).
inline int ln_parts(long long rows, int cols)
{
    int per = 1;
    with_row_shape(cols, [&](auto t, auto) {
        if constexpr (decltype(t)::value > 0)
            per = row_threads(decltype(t)::value) / decltype(t)::value;
    });
    const long long groups = (rows + per - 1) / per;
    if (groups <= 4)
        return 1;
    const int most = cols <= 2048 || cols > 8192 ? 512 : 256;
    return (int)(groups < most ? groups : most);
}

}  // namespace convimg
