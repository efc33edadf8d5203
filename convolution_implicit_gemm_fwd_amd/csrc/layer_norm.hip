// layer_norm.hip -- layer normalisation over the channels of NHWC maps (or
// the columns of token rows), its gradient, and the forward pass that writes
// MXFP4 rows for the quantised linear layer.
//
// With mu, r = mean(x), 1 / sqrt(var(x) + eps) of a row (var over all its
// columns, no correction) and n = (x - mu) r:
//
//   y  = n gamma + beta
//   dx = r (h - mean(h) - n mean(h n)),  h = dy gamma
//   dgamma = sum over rows of dy n,  dbeta = sum over rows of dy
//
// All statistics and sums are fp32.  The variance is taken from the
// differences to the mean, a second pass over the row, so that rows whose
// mean is large against their spread keep their precision.
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

struct LnFwdArgs {
    const void *x;
    const float *gamma, *beta;
    void *y;
    unsigned *scales;      // MXFP4 output: y holds the codes
    float *mean, *rstd;
    long long rows, ldx;
    int cols;
    float eps;
};

// Writes eight normalised values of a row: of type Y, or as MXFP4, whose
// blocks and scale dwords are held by W = 4, 8 or 16 neighbouring lanes, which
// all reach this together.
template <typename Y, int W>
__device__ __forceinline__ void ln_emit(const LnFwdArgs &a, long long row, int col, const float (&v)[8])
{
    if constexpr (__is_same(Y, Mx4)) {
        unsigned top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top = mx_top(top, v[e]);
        const unsigned byte = mx_scale_byte(quad_max(top));
        const int kp = (a.cols + 31) & ~31;
        if (col < kp)
            ((unsigned *)a.y)[row * (kp / 8) + col / 8] = mx_encode8(v, mx_scale_value(byte));
        const unsigned word = mx_scale_word<W>(byte, col >> 5);
        if ((col & 127) == 0 && col < kp)
            a.scales[(long long)(col >> 7) * a.rows + row] = word;
    } else if (col < a.cols) {
        store8<Y>((typename Y::raw *)a.y + row * a.cols, col, a.cols, v);
    }
}

__device__ __forceinline__ void ln_affine(const LnFwdArgs &a, int col, float mean, float rstd, float (&v)[8])
{
    float g[8], b[8];
    if (a.gamma)
        load8<Fp32>(a.gamma, col, a.cols, g);
    if (a.beta)
        load8<Fp32>(a.beta, col, a.cols, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float t = (v[e] - mean) * rstd;
        if (a.gamma)
            t *= g[e];
        if (a.beta)
            t += b[e];
        v[e] = col + e < a.cols ? t : 0.f;
    }
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

// Rows that fit the registers of TPR threads, 8 V columns each; a workgroup
// takes row_threads(TPR) / TPR rows at once, reads each once, and the next
// ones before it sums the present ones.  Bound by memory: 16384 x 4096 bf16
// 43.9 us, 6.1 TB/s (part of it from the memory-side cache), 16384 x 8192
// 100 us, 5.3 TB/s, where a copy of 256 MiB reaches 5.2 to 5.5; a workgroup a
// row without the next row in flight took 68.5 and 161 us.  With MXFP4 rows as
// output 16384 x 4096 takes 45 us, 3.7 TB/s: as long as the 16-bit output, as
// the reads and the row's sums are the same.
template <typename X, typename Y, int TPR, int V>
__global__ __launch_bounds__(row_threads(TPR)) void ln_fwd_rows(LnFwdArgs a)
{
    __shared__ float lds[2][16];
    constexpr int RPB = row_threads(TPR) / TPR;
    constexpr bool WINDOW = TPR > 4 && !__is_same(Y, Mx4);
    const int l = threadIdx.x % TPR;
    const float inv = 1.f / (float)a.cols;
    const RowCols<TPR, V, WINDOW> at(l, a.cols);
    float gm[V][8], bt[V][8];
    Raw8<X> raw[V];
    const long long step = (long long)gridDim.x * RPB;
    // (MXFP4: neighbouring rows' scales share cache lines, so their workgroups
    // share an XCD, of the 8 that take workgroups in turn; the grid is then a
    // multiple of 8)
    const unsigned place = __is_same(Y, Mx4) ? (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3) : blockIdx.x;
    long long row = (long long)place * RPB + threadIdx.x / TPR;
    auto fetch = [&](long long r) {
        if (r < a.rows)
#pragma unroll
            for (int i = 0; i < V; ++i)
                raw[i] = at.template load<X>((const typename X::raw *)a.x + r * a.ldx, i, a.cols);
    };
    fetch(row);
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            gm[i][e] = 1.f;
            bt[i][e] = 0.f;
        }
        if (a.gamma)
            at.template unpack<Fp32>(at.template load<Fp32>(a.gamma, i, a.cols), i, a.cols, gm[i]);
        if (a.beta)
            at.template unpack<Fp32>(at.template load<Fp32>(a.beta, i, a.cols), i, a.cols, bt[i]);
    }
    for (; row < a.rows; row += step) {
        float v[V][8], s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            at.template unpack<X>(raw[i], i, a.cols, v[i]);
        fetch(row + step);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s += !WINDOW || at.counts(i, e) ? v[i][e] : 0.f;
        const float mean = row_sum<TPR>(s, lds[0]) * inv;
        s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[i][e] = WINDOW || at.col[i] + e < a.cols ? v[i][e] - mean : 0.f;
                s += !WINDOW || at.counts(i, e) ? v[i][e] * v[i][e] : 0.f;
            }
        const float rstd = 1.f / sqrtf(row_sum<TPR>(s, lds[1]) * inv + a.eps);
        if (l == 0) {
            if (a.mean)
                a.mean[row] = mean;
            if (a.rstd)
                a.rstd[row] = rstd;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            // (in MXFP4's last block v, beta and so the result are 0 past the row)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[i][e] = v[i][e] * rstd * gm[i][e] + bt[i][e];
            ln_emit<Y, (TPR < 16 ? TPR : 16)>(a, row, at.col[i], v[i]);
        }
    }
}

// One workgroup a row, for rows past 8192 columns, which the registers of 1024
// threads do not hold at eight each: the row is read three times (mean,
// variance, result), the later ones from cache in part.  4096 x 12288 bf16 67 us
// (195 MB read and 101 written, 3.0 TB/s of the 201 MB that it needs), 4096 x
// 16384 93 us; with MXFP4 rows as output 60 and 80 us.
template <typename X, typename Y>
__global__ __launch_bounds__(kLnThreads) void ln_fwd_wide(LnFwdArgs a)
{
    __shared__ float lds[4];
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const typename X::raw *x = (const typename X::raw *)a.x + row * a.ldx;
        float v[8], s = 0.f;
        for (int c = threadIdx.x * 8; c < a.cols; c += kLnThreads * 8) {
            load8<X>(x, c, a.cols, v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s += v[e];
        }
        const float mean = block_sum(s, lds) / (float)a.cols;
        s = 0.f;
        for (int c = threadIdx.x * 8; c < a.cols; c += kLnThreads * 8) {
            load8<X>(x, c, a.cols, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = c + e < a.cols ? v[e] - mean : 0.f;
                s += d * d;
            }
        }
        const float rstd = 1.f / sqrtf(block_sum(s, lds) / (float)a.cols + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean)
                a.mean[row] = mean;
            if (a.rstd)
                a.rstd[row] = rstd;
        }
        // whole runs of 128 columns, so that the lanes of a scale dword stay together
        const int end = (a.cols + 127) & ~127;
        for (int c = threadIdx.x * 8; c < end; c += kLnThreads * 8) {
            load8<X>(x, c, a.cols, v);
            ln_affine(a, c, mean, rstd, v);
            ln_emit<Y, 16>(a, row, c, v);
        }
    }
}

struct LnBwdArgs {
    const void *dy, *x;
    const float *gamma, *mean, *rstd;
    void *dx;
    float *part_g, *part_b;      // sums of dy n and of dy, a row of `cols` every part_ld floats; NULL to skip them
    long long part_ld;
    long long rows, lddy, ldx;
    int cols, dx_dtype, parts;
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

// The input's gradient for rows past 8192 columns, one workgroup a row: the
// row's two sums, then dx, each from a read of dy and x.  4096 x 12288 bf16 79
// us of the 139 that the whole gradient takes (403 MB read and 101 written).
template <typename DY, typename X>
__global__ __launch_bounds__(kLnThreads) void ln_bwd_dx_wide(LnBwdArgs a)
{
    __shared__ float lds[4];
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const typename X::raw *x = (const typename X::raw *)a.x + row * a.ldx;
        const typename DY::raw *dy = (const typename DY::raw *)a.dy + row * a.lddy;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s1 = 0.f, s2 = 0.f;
        for (int c = threadIdx.x * 8; c < a.cols; c += kLnThreads * 8) {
            float n[8], h[8], g[8];
            load8<X>(x, c, a.cols, n);
            load8<DY>(dy, c, a.cols, h);
            if (a.gamma)
                load8<Fp32>(a.gamma, c, a.cols, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float t = a.gamma ? h[e] * g[e] : h[e];
                s1 += t;
                s2 += c + e < a.cols ? t * ((n[e] - mean) * rstd) : 0.f;
            }
        }
        const float m1 = block_sum(s1, lds) / (float)a.cols;
        const float m2 = block_sum(s2, lds) / (float)a.cols;
        for (int c = threadIdx.x * 8; c < a.cols; c += kLnThreads * 8) {
            float n[8], h[8], g[8];
            load8<X>(x, c, a.cols, n);
            load8<DY>(dy, c, a.cols, h);
            if (a.gamma)
                load8<Fp32>(a.gamma, c, a.cols, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float t = a.gamma ? h[e] * g[e] : h[e];
                h[e] = rstd * (t - m1 - ((n[e] - mean) * rstd) * m2);
            }
            store8_as(a.dx_dtype, a.dx, row, c, a.cols, h);
        }
    }
}

// Partial sums for the parameters' gradients of such rows: a thread owns
// eight columns and walks every parts-th row (4096 x 12288 40 us, 202 MB read
// and 50 written, and 17 us for the sums over them).
template <typename DY, typename X>
__global__ __launch_bounds__(kLnThreads) void ln_bwd_cols_wide(LnBwdArgs a)
{
    const int c = (blockIdx.x * kLnThreads + threadIdx.x) * 8;
    if (c >= a.cols)
        return;
    float dg[8] = {}, db[8] = {};
    for (long long row = blockIdx.y; row < a.rows; row += a.parts) {
        float n[8], h[8];
        load8<X>((const typename X::raw *)a.x + row * a.ldx, c, a.cols, n);
        load8<DY>((const typename DY::raw *)a.dy + row * a.lddy, c, a.cols, h);
        const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dg[e] += h[e] * ((n[e] - mean) * rstd);
            db[e] += h[e];
        }
    }
    store8<Fp32>(a.part_g + blockIdx.y * a.part_ld, c, a.cols, dg);
    store8<Fp32>(a.part_b + blockIdx.y * a.part_ld, c, a.cols, db);
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

// The whole gradient in one pass over dy and x, for rows that fit the
// registers of TPR threads (8 V columns each).  A workgroup walks every
// parts-th group of row_threads(TPR) / TPR rows, reads the next group's values
// before it sums the present one's, and keeps its columns' sums of dy n and
// dy in registers; at the end it adds those of its row groups in a fixed
// order and writes one partial sum.  Bound by memory: 16384 x 4096 bf16 74 us
// (403 MB, 5.4 TB/s) and 4.5 us for the partial sums; two passes over dy and x
// took 242 us.
template <typename DY, typename X, int TPR, int V>
__global__ __launch_bounds__(row_threads(TPR)) void ln_bwd_rows(LnBwdArgs a)
{
    constexpr int RPB = row_threads(TPR) / TPR;
    constexpr bool WINDOW = TPR > 4;
    __shared__ float lds[2][16][2];
    __shared__ float sums[TPR > 64 ? 1 : 4][2][TPR > 64 ? 1 : TPR * 8 * V];
    const int l = threadIdx.x % TPR;
    const float inv = 1.f / (float)a.cols;
    const RowCols<TPR, V, WINDOW> at(l, a.cols);
    float gm[V][8], dg[V][8] = {}, db[V][8] = {};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (a.gamma)
            at.template unpack<Fp32>(at.template load<Fp32>(a.gamma, i, a.cols), i, a.cols, gm[i]);
        else
#pragma unroll
            for (int e = 0; e < 8; ++e)
                gm[i][e] = 1.f;
    }
    Raw8<X> rx[V];
    Raw8<DY> rd[V];
    float mean = 0.f, rstd = 0.f;
    const long long step = (long long)a.parts * RPB;
    long long row = (long long)blockIdx.x * RPB + threadIdx.x / TPR;
    auto fetch = [&](long long r) {
        if (r >= a.rows)
            return;
        mean = a.mean[r];
        rstd = a.rstd[r];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            rx[i] = at.template load<X>((const typename X::raw *)a.x + r * a.ldx, i, a.cols);
            rd[i] = at.template load<DY>((const typename DY::raw *)a.dy + r * a.lddy, i, a.cols);
        }
    };
    fetch(row);
    for (int k = 0; row < a.rows; row += step, k ^= 1) {
        float n[V][8], h[V][8], s1 = 0.f, s2 = 0.f;
        const float m = mean, r = rstd;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            at.template unpack<X>(rx[i], i, a.cols, n[i]);
            at.template unpack<DY>(rd[i], i, a.cols, h[i]);
        }
        fetch(row + step);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // (past the row h is 0)
                n[i][e] = WINDOW || at.col[i] + e < a.cols ? (n[i][e] - m) * r : 0.f;
                dg[i][e] += h[i][e] * n[i][e];
                db[i][e] += h[i][e];
                h[i][e] *= gm[i][e];
                s1 += !WINDOW || at.counts(i, e) ? h[i][e] : 0.f;
                s2 += !WINDOW || at.counts(i, e) ? h[i][e] * n[i][e] : 0.f;
            }
        row_sum2<TPR>(s1, s2, lds[k]);
        s1 *= inv;
        s2 *= inv;
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                h[i][e] = r * (h[i][e] - s1 - n[i][e] * s2);
            if (at.col[i] < a.cols)
                store8_as(a.dx_dtype, a.dx, row, at.col[i], a.cols, h[i]);
        }
    }
    if (!a.part_g)
        return;
    float *pg = a.part_g + blockIdx.x * a.part_ld, *pb = a.part_b + blockIdx.x * a.part_ld;
    if constexpr (TPR > 64) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (at.col[i] < a.cols) {
                store8<Fp32>(pg, at.col[i], a.cols, dg[i]);
                store8<Fp32>(pb, at.col[i], a.cols, db[i]);
            }
    } else {
        // the wave's row groups, then the four waves
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float g = stride_sum<TPR>(dg[i][e]), b = stride_sum<TPR>(db[i][e]);
                if ((threadIdx.x & 63) < TPR) {
                    sums[threadIdx.x >> 6][0][at.col[i] + e] = g;
                    sums[threadIdx.x >> 6][1][at.col[i] + e] = b;
                }
            }
        __syncthreads();
        for (int c = threadIdx.x; c < a.cols; c += kLnThreads) {
            pg[c] = (sums[0][0][c] + sums[1][0][c]) + (sums[2][0][c] + sums[3][0][c]);
            pb[c] = (sums[0][1][c] + sums[1][1][c]) + (sums[2][1][c] + sums[3][1][c]);
        }
    }
}

// dgamma and dbeta: the partial sums in a fixed order, 16 columns a workgroup
// and 64 threads a column (512 sums of 128 columns: 3 us; a thread a column took
// 62).  A launch takes the columns from `first`, up to kLnRedStep of the 2
// cols, as it holds fewer than 2^32 threads.
constexpr int kLnRedCols = 16, kLnRedThreads = 1024, kLnRedStep = 1 << 24;

__global__ __launch_bounds__(kLnRedThreads) void ln_bwd_reduce(const float *part, float *dgamma, float *dbeta,
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

// Rows and columns each fit an int; all element offsets are 64-bit.
int ln_check(const void *x, long long ldx, long long rows, int cols, int dtype)
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
unsigned ln_grid(long long rows) { return (unsigned)(rows < (1 << 22) ? rows : (1 << 22)); }

// Workgroups of the forward pass: at most what 256 CUs hold of 2048 threads,
// which walk the rows.
unsigned ln_fwd_grid(long long rows, int tpr, bool eights)
{
    const long long per = row_threads(tpr) / tpr, n = (rows + per - 1) / per;
    const long long most = 256 * 2048 / row_threads(tpr);
    const unsigned g = (unsigned)(n < most ? n : most);
    return eights ? (g + 7) & ~7u : g;
}

template <typename X, typename Y>
void ln_fwd_launch(const LnFwdArgs &a, hipStream_t stream)
{
    with_row_shape(a.cols, [&](auto t, auto v) {
        constexpr int TPR = decltype(t)::value, V = decltype(v)::value;
        if constexpr (TPR == 0)
            hipLaunchKernelGGL((ln_fwd_wide<X, Y>), dim3(ln_grid(a.rows)), dim3(kLnThreads), 0, stream, a);
        else
            hipLaunchKernelGGL((ln_fwd_rows<X, Y, TPR, V>), dim3(ln_fwd_grid(a.rows, TPR, std::is_same<Y, Mx4>::value)),
                               dim3(row_threads(TPR)), 0, stream, a);
    });
}

int ln_fwd_call(const LnFwdArgs &a, int x_dtype, int y_dtype, hipStream_t stream)
{
    const size_t nx = span_bytes(a.rows, a.ldx, a.cols, x_dtype);
    const size_t ny = a.scales ? mx_code_bytes(a.rows, a.cols) : span_bytes(a.rows, a.cols, a.cols, y_dtype);
    const size_t ns = a.scales ? mx_scale_bytes(a.rows, a.cols) : 0;
    const size_t np = (size_t)a.cols * 4, nr = (size_t)a.rows * 4;
    const void *out[4] = {a.y, a.scales, a.mean, a.rstd};
    const size_t nout[4] = {ny, ns, nr, nr};
    for (int i = 0; i < 4; ++i) {
        if (row_overlaps(out[i], nout[i], a.x, nx) || row_overlaps(out[i], nout[i], a.gamma, np)
            || row_overlaps(out[i], nout[i], a.beta, np))
            return CONVIMG_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (row_overlaps(out[i], nout[i], out[j], nout[j]))
                return CONVIMG_ERR_ALIAS;
    }
    if (a.rows == 0)
        return CONVIMG_OK;
    with_dtype(x_dtype, [&](auto x) {
        if (a.scales)
            ln_fwd_launch<decltype(x), Mx4>(a, stream);
        else
            with_dtype(y_dtype, [&](auto y) { ln_fwd_launch<decltype(x), decltype(y)>(a, stream); });
    });
    return hipGetLastError() == hipSuccess ? CONVIMG_OK : CONVIMG_ERR_LAUNCH;
}

// Partial sums of the parameters' gradients, one a workgroup of the
// backward pass: enough workgroups to keep the memory busy, few enough that
// the partial sums (2 cols fp32 each, written and read) stay small beside
// dy, x and dx.  A single one writes the gradients itself: so do up to four
// groups of rows, for which a second launch (4 us) would cost more than the
// other workgroups save.  512 workgroups of 256 threads, 256 of more (65536 x
// 128 16.9 us, 17.8 with 1024; 65536 x 1024 75 us, 88 with 1024; 16384 x 4096
// 79 us, 81 with 512; 8192 x 8192 81 us, 91 with 512).
int ln_parts(long long rows, int cols)
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

template <typename DY, typename X>
void ln_bwd_launch(const LnBwdArgs &a, hipStream_t stream)
{
    with_row_shape(a.cols, [&](auto t, auto v) {
        constexpr int TPR = decltype(t)::value, V = decltype(v)::value;
        if constexpr (TPR == 0) {
            if (a.rows > 0)
                hipLaunchKernelGGL((ln_bwd_dx_wide<DY, X>), dim3(ln_grid(a.rows)), dim3(kLnThreads),
                                   0, stream, a);
            if (a.part_g)
                hipLaunchKernelGGL((ln_bwd_cols_wide<DY, X>),
                                   dim3((a.cols + 8 * kLnThreads - 1) / (8 * kLnThreads), a.parts), dim3(kLnThreads),
                                   0, stream, a);
        } else {
            hipLaunchKernelGGL((ln_bwd_rows<DY, X, TPR, V>), dim3(a.parts), dim3(row_threads(TPR)), 0, stream, a);
        }
    });
}

}  // namespace convimg

using namespace convimg;

extern "C" {

int layer_norm_fwd(const void *x, long long ldx, const float *gamma, const float *beta, long long rows, int cols,
                   float eps, int x_dtype, int y_dtype, void *y, float *mean, float *rstd, hipStream_t stream)
{
    const int rc = ln_check(x, ldx, rows, cols, x_dtype);
    if (rc != CONVIMG_OK)
        return rc;
    if (!dtype_ok(y_dtype))
        return CONVIMG_ERR_DTYPE;
    if (!y && rows > 0)
        return CONVIMG_ERR_NULL;
    const LnFwdArgs a = {x, gamma, beta, y, nullptr, mean, rstd, rows, ldx, cols, eps};
    return ln_fwd_call(a, x_dtype, y_dtype, stream);
}

int layer_norm_fwd_mxfp4(const void *x, long long ldx, const float *gamma, const float *beta, long long rows,
                         int cols, float eps, int x_dtype, void *codes, void *scales, float *mean, float *rstd,
                         hipStream_t stream)
{
    int rc = ln_check(x, ldx, rows, cols, x_dtype);
    if (rc == CONVIMG_OK)
        rc = mx_shape(rows, cols);
    if (rc != CONVIMG_OK)
        return rc;
    if (rows == 0)
        return CONVIMG_OK;
    if (!codes || !scales)
        return CONVIMG_ERR_NULL;
    if (((uintptr_t)codes & 15) || ((uintptr_t)scales & 3))
        return CONVIMG_ERR_ALIGN;
    const LnFwdArgs a = {x, gamma, beta, codes, (unsigned *)scales, mean, rstd, rows, ldx, cols, eps};
    return ln_fwd_call(a, x_dtype, CONVIMG_BF16, stream);
}

int layer_norm_bwd_workspace(long long rows, int cols, size_t *bytes)
{
    if (!bytes)
        return CONVIMG_ERR_NULL;
    if (rows < 0 || cols <= 0)
        return CONVIMG_ERR_SHAPE;
    if (rows > kMaxRows || cols > kMaxCols)
        return CONVIMG_ERR_RANGE;
    *bytes = (size_t)ln_parts(rows, cols) * 2 * (size_t)cols * 4;
    return CONVIMG_OK;
}

int layer_norm_bwd(const void *dy, long long lddy, const void *x, long long ldx, const float *gamma,
                   const float *mean, const float *rstd, long long rows, int cols, int dy_dtype, int x_dtype,
                   int dx_dtype, void *dx, float *dgamma, float *dbeta, void *ws, size_t ws_bytes,
                   hipStream_t stream)
{
    int rc = ln_check(x, ldx, rows, cols, x_dtype);
    if (rc == CONVIMG_OK)
        rc = ln_check(dy, lddy, rows, cols, dy_dtype);
    if (rc != CONVIMG_OK)
        return rc;
    if (!dtype_ok(dx_dtype))
        return CONVIMG_ERR_DTYPE;
    if ((rows > 0 && (!dx || !mean || !rstd)) || (!dgamma) != (!dbeta))
        return CONVIMG_ERR_NULL;
    size_t need = 0;
    (void)layer_norm_bwd_workspace(rows, cols, &need);
    if (!dgamma)
        need = 0;
    if (need > 0 && !ws)
        return CONVIMG_ERR_NULL;
    if (need > 0 && ((uintptr_t)ws & 15))
        return CONVIMG_ERR_ALIGN;
    if (ws_bytes < need)
        return CONVIMG_ERR_WORKSPACE;
    const size_t np = (size_t)cols * 4, nr = (size_t)rows * 4;
    const void *in[5] = {dy, x, gamma, mean, rstd};
    const size_t nin[5] = {span_bytes(rows, lddy, cols, dy_dtype), span_bytes(rows, ldx, cols, x_dtype), np, nr, nr};
    const void *out[4] = {dx, dgamma, dbeta, need ? ws : nullptr};
    const size_t nout[4] = {span_bytes(rows, cols, cols, dx_dtype), np, np, need};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 5; ++j)
            if (row_overlaps(out[i], nout[i], in[j], nin[j]))
                return CONVIMG_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (row_overlaps(out[i], nout[i], out[j], nout[j]))
                return CONVIMG_ERR_ALIAS;
    }
    const int parts = ln_parts(rows, cols);
    float *pg = parts > 1 && dgamma ? (float *)ws : dgamma, *pb = parts > 1 && dgamma ? pg + cols : dbeta;
    const LnBwdArgs a = {dy,   x,    gamma, mean, rstd,     dx,   pg,   pb, 2LL * cols,
                         rows, lddy, ldx,   cols, dx_dtype, parts};
    if (rows == 0 && !dgamma)
        return CONVIMG_OK;
    // (with no rows the one sum is 0)
    with_dtype(dy_dtype, [&](auto d) {
        with_dtype(x_dtype, [&](auto t) { ln_bwd_launch<decltype(d), decltype(t)>(a, stream); });
    });
    if (dgamma && parts > 1)
        for (long long c = 0, end = 2LL * cols; c < end; c += kLnRedStep) {
            const long long n = end - c < kLnRedStep ? end - c : kLnRedStep;
            hipLaunchKernelGGL(ln_bwd_reduce, dim3((unsigned)((n + kLnRedCols - 1) / kLnRedCols)), dim3(kLnRedThreads), 0,
                               stream, pg, dgamma, dbeta, cols, parts, c);
        }
    return hipGetLastError() == hipSuccess ? CONVIMG_OK : CONVIMG_ERR_LAUNCH;
}

}  // extern "C"
