// layer_norm_kept.hip -- layer normalisation that keeps n = (x - mu) r in 8
// bits for its gradient (mxint8.hpp), and the gradient from that:
//
//   y  = n gamma + beta
//   dx = r (h - mean(h) - n mean(h n)),  h = dy gamma
//   dgamma = sum over rows of dy n,  dbeta = sum over rows of dy
//
// The backward pass needs neither x nor mu, and n is of one size in every row,
// however far a row's mean lies from its spread.  Statistics and sums are fp32;
// the one rounding to 8 bits is that of the kept n, y is taken from n before it.
//
// Memory bounds both.  Forward, 50176 x 64 from fp32 to bf16: 7.3 us (23 MB);
// 16384 x 4096 in bf16 68 us (337 MB, 5.0 TB/s).  Past 8192 columns, where x is read
// three times forward, dy and the codes three times backward: 8192 x 10000 in bf16
// 138 us (412 MB, 3.0 TB/s) and 122 + 52 + 14.
// Backward, 16384 x 4096 in bf16: 72.5 us (347 MB, 4.8 TB/s; from x, mu and r
// 75.0), 5.0 more for the sums over the 256 workgroups' partial sums.
#include "layer_norm.hpp"
#include "mxint8.hpp"

namespace convimg {

struct LnKeptArgs {
    const void *x;
    const float *gamma, *beta;
    void *y;
    unsigned char *codes;
    unsigned *scales;
    float *rstd;
    long long rows, ldx;
    int cols, y_dtype;
    float eps;
};

// Rows that fit the registers of TPR threads, 8 V columns each, with the next
// row in flight (as the forward pass that keeps nothing).  Columns stay at
// their places, unlike there, so that four lanes hold a block.
template <typename X, int TPR, int V>
__global__ __launch_bounds__(row_threads(TPR)) void ln_kept_rows(LnKeptArgs a)
{
    __shared__ float lds[2][16];
    constexpr int RPB = row_threads(TPR) / TPR;
    const int l = threadIdx.x % TPR;
    const RowCols<TPR, V, false> at(l, a.cols);
    float gm[V][8], bt[V][8];
    Raw8<X> raw[V];
    const long long step = (long long)gridDim.x * RPB;
    long long row = (long long)blockIdx.x * RPB + threadIdx.x / TPR;
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
                s += v[i][e];
        // (divided, not multiplied by 1 / cols: where the sum is exact a constant
        // row's mean is then its value, and n exactly 0)
        const float mean = row_sum<TPR>(s, lds[0]) / (float)a.cols;
        s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[i][e] = at.col[i] + e < a.cols ? v[i][e] - mean : 0.f;
                s += v[i][e] * v[i][e];
            }
        const float rstd = 1.f / sqrtf(row_sum<TPR>(s, lds[1]) / (float)a.cols + a.eps);
        if (l == 0)
            a.rstd[row] = rstd;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            // (past the row n stays 0 where rstd is infinite, too)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[i][e] = at.col[i] + e < a.cols ? v[i][e] * rstd : 0.f;
            mxi_emit8<(TPR < 16 ? TPR : 16)>(a.codes, a.scales, row, a.cols, at.col[i], v[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[i][e] = v[i][e] * gm[i][e] + bt[i][e];
            if (at.col[i] < a.cols)
                store8_as(a.y_dtype, a.y, row, at.col[i], a.cols, v[i]);
        }
    }
}

// One workgroup a row, for rows past 8192 columns: the row is read three
// times, the later ones from cache in part.
template <typename X>
__global__ __launch_bounds__(kLnThreads) void ln_kept_wide(LnKeptArgs a)
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
        if (threadIdx.x == 0)
            a.rstd[row] = rstd;
        // whole runs of 128 columns, so that the lanes of a scale dword stay together
        const int end = (a.cols + 127) & ~127;
        for (int c = threadIdx.x * 8; c < end; c += kLnThreads * 8) {
            load8<X>(x, c, a.cols, v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = c + e < a.cols ? (v[e] - mean) * rstd : 0.f;
            mxi_emit8<16>(a.codes, a.scales, row, a.cols, c, v);
            if (c >= a.cols)
                continue;
            float g[8], b[8];
            if (a.gamma)
                load8<Fp32>(a.gamma, c, a.cols, g);
            if (a.beta)
                load8<Fp32>(a.beta, c, a.cols, b);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = (a.gamma ? v[e] * g[e] : v[e]) + (a.beta ? b[e] : 0.f);
            store8_as(a.y_dtype, a.y, row, c, a.cols, v);
        }
    }
}

struct LnKeptBwdArgs {
    const void *dy;
    const unsigned char *codes, *scales;
    const float *gamma, *rstd;
    void *dx;
    float *part_g, *part_b;      // sums of dy n and of dy, a row of `cols` every part_ld floats; NULL to skip them
    long long part_ld;
    long long rows, lddy;
    int cols, dx_dtype, parts;
};

// Eight kept values from any column on; with WINDOW they may lie in two blocks.
template <bool WINDOW>
struct Kept8 {
    unsigned q[2], byte[WINDOW ? 2 : 1];

    __device__ __forceinline__ void load(const LnKeptBwdArgs &a, long long row, int col)
    {
        typedef unsigned u32v2 __attribute__((ext_vector_type(2)));
        typedef u32v2 u32v2_a1 __attribute__((aligned(1)));
        if (col >= a.cols)
            return;
        const int kp = (a.cols + 31) & ~31;
        const unsigned char *s = a.scales + row * (((a.cols + 127) >> 7) * 4);
        const u32v2 v = *(const u32v2_a1 *)(a.codes + row * kp + col);
        q[0] = v[0];
        q[1] = v[1];
        byte[0] = s[col >> 5];
        if constexpr (WINDOW)
            byte[1] = s[(col + 7) >> 5];
    }
    __device__ __forceinline__ void unpack(int col, float (&v)[8]) const
    {
        if constexpr (WINDOW) {
            const float u0 = mx_scale_value(byte[0]), u1 = mx_scale_value(byte[1]);
            const int first = 32 - (col & 31);      // of the second block
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = (float)(signed char)(q[e / 4] >> (8 * (e & 3))) * (e < first ? u0 : u1);
        } else {
            mxi_decode8(uint2{q[0], q[1]}, mx_scale_value(byte[0]), v);
        }
    }
};

// The whole gradient in one pass, for rows that fit the registers of TPR
// threads; a workgroup walks every parts-th group of rows with the next one in
// flight and keeps its columns' sums in registers.
template <typename DY, int TPR, int V>
__global__ __launch_bounds__(row_threads(TPR)) void ln_kept_bwd_rows(LnKeptBwdArgs a)
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
    Kept8<WINDOW> rx[V] = {};
    Raw8<DY> rd[V];
    float rstd = 0.f;
    const long long step = (long long)a.parts * RPB;
    long long row = (long long)blockIdx.x * RPB + threadIdx.x / TPR;
    auto fetch = [&](long long r) {
        if (r >= a.rows)
            return;
        rstd = a.rstd[r];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            rx[i].load(a, r, at.col[i]);
            rd[i] = at.template load<DY>((const typename DY::raw *)a.dy + r * a.lddy, i, a.cols);
        }
    };
    fetch(row);
    for (int k = 0; row < a.rows; row += step, k ^= 1) {
        float n[V][8], h[V][8], s1 = 0.f, s2 = 0.f;
        const float r = rstd;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            rx[i].unpack(at.col[i], n[i]);
            at.template unpack<DY>(rd[i], i, a.cols, h[i]);
        }
        fetch(row + step);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // (past the row h is 0)
                n[i][e] = WINDOW || at.col[i] + e < a.cols ? n[i][e] : 0.f;
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

// The input's gradient for rows past 8192 columns, one workgroup a row.
template <typename DY>
__global__ __launch_bounds__(kLnThreads) void ln_kept_bwd_dx_wide(LnKeptBwdArgs a)
{
    __shared__ float lds[4];
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const typename DY::raw *dy = (const typename DY::raw *)a.dy + row * a.lddy;
        const float rstd = a.rstd[row];
        float s1 = 0.f, s2 = 0.f, n[8], h[8], g[8];
        auto get = [&](int c) {
            Kept8<false> k;
            k.load(a, row, c);
            k.unpack(c, n);
            load8<DY>(dy, c, a.cols, h);
            if (a.gamma)
                load8<Fp32>(a.gamma, c, a.cols, g);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                h[e] = a.gamma ? h[e] * g[e] : h[e];
        };
        for (int c = threadIdx.x * 8; c < a.cols; c += kLnThreads * 8) {
            get(c);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s1 += h[e];
                s2 += c + e < a.cols ? h[e] * n[e] : 0.f;
            }
        }
        const float m1 = block_sum(s1, lds) / (float)a.cols;
        const float m2 = block_sum(s2, lds) / (float)a.cols;
        for (int c = threadIdx.x * 8; c < a.cols; c += kLnThreads * 8) {
            get(c);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                h[e] = rstd * (h[e] - m1 - n[e] * m2);
            store8_as(a.dx_dtype, a.dx, row, c, a.cols, h);
        }
    }
}

// Partial sums for the parameters' gradients of such rows: a thread owns
// eight columns and walks every parts-th row.
template <typename DY>
__global__ __launch_bounds__(kLnThreads) void ln_kept_bwd_cols_wide(LnKeptBwdArgs a)
{
    const int c = (blockIdx.x * kLnThreads + threadIdx.x) * 8;
    if (c >= a.cols)
        return;
    float dg[8] = {}, db[8] = {};
    for (long long row = blockIdx.y; row < a.rows; row += a.parts) {
        float n[8], h[8];
        Kept8<false> k;
        k.load(a, row, c);
        k.unpack(c, n);
        load8<DY>((const typename DY::raw *)a.dy + row * a.lddy, c, a.cols, h);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dg[e] += h[e] * n[e];
            db[e] += h[e];
        }
    }
    store8<Fp32>(a.part_g + blockIdx.y * a.part_ld, c, a.cols, dg);
    store8<Fp32>(a.part_b + blockIdx.y * a.part_ld, c, a.cols, db);
}

template <typename DY>
void ln_kept_bwd_launch(const LnKeptBwdArgs &a, hipStream_t stream)
{
    with_row_shape(a.cols, [&](auto t, auto v) {
        constexpr int TPR = decltype(t)::value, V = decltype(v)::value;
        if constexpr (TPR == 0) {
            if (a.rows > 0)
                hipLaunchKernelGGL(ln_kept_bwd_dx_wide<DY>, dim3(ln_grid(a.rows)), dim3(kLnThreads), 0, stream, a);
            if (a.part_g)
                hipLaunchKernelGGL(ln_kept_bwd_cols_wide<DY>,
                                   dim3((a.cols + 8 * kLnThreads - 1) / (8 * kLnThreads), a.parts), dim3(kLnThreads), 0,
                                   stream, a);
        } else {
            hipLaunchKernelGGL((ln_kept_bwd_rows<DY, TPR, V>), dim3(a.parts), dim3(row_threads(TPR)), 0, stream, a);
        }
    });
}

bool kept_misaligned(const void *codes, const void *scales) { return ((uintptr_t)codes & 15) || ((uintptr_t)scales & 3); }

}  // namespace convimg

using namespace convimg;

extern "C" {

int layer_norm_fwd_mxint8(const void *x, long long ldx, const float *gamma, const float *beta, long long rows,
                          int cols, float eps, int x_dtype, int y_dtype, void *y, void *codes, void *scales,
                          float *rstd, hipStream_t stream)
{
    const int rc = ln_check(x, ldx, rows, cols, x_dtype);
    if (rc != CONVIMG_OK)
        return rc;
    if (!dtype_ok(y_dtype))
        return CONVIMG_ERR_DTYPE;
    if (rows == 0)
        return CONVIMG_OK;
    if (!y || !codes || !scales || !rstd)
        return CONVIMG_ERR_NULL;
    if (kept_misaligned(codes, scales))
        return CONVIMG_ERR_ALIGN;
    const void *in[3] = {x, gamma, beta}, *out[4] = {y, codes, scales, rstd};
    const size_t np = (size_t)cols * 4, nin[3] = {span_bytes(rows, ldx, cols, x_dtype), np, np},
                 nout[4] = {span_bytes(rows, cols, cols, y_dtype), mxi_code_bytes(rows, cols), mxi_scale_bytes(rows, cols),
                            (size_t)rows * 4};
    if (any_overlap(out, nout, 4, in, nin, 3))
        return CONVIMG_ERR_ALIAS;
    const LnKeptArgs a = {x,    gamma, beta, y,       (unsigned char *)codes, (unsigned *)scales, rstd,
                          rows, ldx,   cols, y_dtype, eps};
    with_dtype(x_dtype, [&](auto t) {
        typedef decltype(t) X;
        with_row_shape(cols, [&](auto n, auto v) {
            constexpr int TPR = decltype(n)::value, V = decltype(v)::value;
            if constexpr (TPR == 0)
                hipLaunchKernelGGL(ln_kept_wide<X>, dim3(ln_grid(rows)), dim3(kLnThreads), 0, stream, a);
            else
                hipLaunchKernelGGL((ln_kept_rows<X, TPR, V>), dim3(ln_fwd_grid(rows, TPR, false)), dim3(row_threads(TPR)),
                                   0, stream, a);
        });
    });
    return hipGetLastError() == hipSuccess ? CONVIMG_OK : CONVIMG_ERR_LAUNCH;
}

int layer_norm_bwd_mxint8(const void *dy, long long lddy, const void *codes, const void *scales, const float *gamma,
                          const float *rstd, long long rows, int cols, int dy_dtype, int dx_dtype, void *dx,
                          float *dgamma, float *dbeta, void *ws, size_t ws_bytes, hipStream_t stream)
{
    const int rc = ln_check(dy, lddy, rows, cols, dy_dtype);
    if (rc != CONVIMG_OK)
        return rc;
    if (!dtype_ok(dx_dtype))
        return CONVIMG_ERR_DTYPE;
    if ((rows > 0 && (!dx || !codes || !scales || !rstd)) || (!dgamma) != (!dbeta))
        return CONVIMG_ERR_NULL;
    size_t need = 0;
    (void)layer_norm_bwd_workspace(rows, cols, &need);
    if (!dgamma)
        need = 0;
    if (need > 0 && !ws)
        return CONVIMG_ERR_NULL;
    if ((need > 0 && ((uintptr_t)ws & 15)) || kept_misaligned(codes, scales))
        return CONVIMG_ERR_ALIGN;
    if (ws_bytes < need)
        return CONVIMG_ERR_WORKSPACE;
    const size_t np = (size_t)cols * 4;
    const void *in[5] = {dy, codes, scales, gamma, rstd}, *out[4] = {dx, dgamma, dbeta, need ? ws : nullptr};
    const size_t nin[5] = {span_bytes(rows, lddy, cols, dy_dtype), mxi_code_bytes(rows, cols), mxi_scale_bytes(rows, cols),
                           np, (size_t)rows * 4},
                 nout[4] = {span_bytes(rows, cols, cols, dx_dtype), np, np, need};
    if (any_overlap(out, nout, 4, in, nin, 5))
        return CONVIMG_ERR_ALIAS;
    const int parts = ln_parts(rows, cols);
    float *pg = parts > 1 && dgamma ? (float *)ws : dgamma, *pb = parts > 1 && dgamma ? pg + cols : dbeta;
    const LnKeptBwdArgs a = {dy, (const unsigned char *)codes, (const unsigned char *)scales, gamma, rstd, dx, pg, pb,
                             2LL * cols, rows, lddy, cols, dx_dtype, parts};
    if (rows == 0 && !dgamma)
        return CONVIMG_OK;
    // (with no rows the one sum is 0)
    with_dtype(dy_dtype, [&](auto d) { ln_kept_bwd_launch<decltype(d)>(a, stream); });
    if (dgamma && parts > 1)
        ln_reduce_parts(pg, dgamma, dbeta, cols, parts, stream);
    return hipGetLastError() == hipSuccess ? CONVIMG_OK : CONVIMG_ERR_LAUNCH;
}

}  // extern "C"
