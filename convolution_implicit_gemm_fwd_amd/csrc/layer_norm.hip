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

struct Mx4 {};

// Writes eight normalised values of a row: of type Y, or as MXFP4 (four
// neighbouring lanes hold one block; all of them reach this together).
template <typename Y>
__device__ __forceinline__ void ln_emit(const LnFwdArgs &a, long long row, int col, const float (&v)[8])
{
    if constexpr (__is_same(Y, Mx4)) {
        unsigned top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top = mx_top(top, v[e]);
        top = max(top, (unsigned)__shfl_xor((int)top, 1, 64));
        top = max(top, (unsigned)__shfl_xor((int)top, 2, 64));
        const unsigned byte = mx_scale_byte(top);
        const int kp = (a.cols + 31) & ~31;
        if (col < kp) {
            ((unsigned *)a.y)[row * (kp / 8) + col / 8] = mx_encode8(v, mx_scale_value(byte));
            unsigned char *s = (unsigned char *)(a.scales + (long long)(col >> 7) * a.rows + row);
            if ((col & 31) == 0) {
                s[(col >> 5) & 3] = (unsigned char)byte;
                // bytes of blocks past the row's last one are 0
                if (col + 32 == kp)
                    for (int b = ((col >> 5) & 3) + 1; b < 4; ++b)
                        s[b] = 0;
            }
        }
    } else {
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

// One workgroup a row, any width: the row is read three times (mean,
// variance, result).
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
        // whole blocks of 32 columns, so that the lanes of a block stay together
        const int kp = (a.cols + 31) & ~31;
        for (int c = threadIdx.x * 8; c < kp; c += kLnThreads * 8) {
            load8<X>(x, c, a.cols, v);
            ln_affine(a, c, mean, rstd, v);
            ln_emit<Y>(a, row, c, v);
        }
    }
}

struct LnBwdArgs {
    const void *dy, *x;
    const float *gamma, *mean, *rstd;
    void *dx;
    float *part;           // [parts][2][cols]: sums of dy n and of dy
    float *dgamma, *dbeta;
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

// The input's gradient, one workgroup a row, any width: the row's two sums,
// then dx.
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

// Partial sums over a range of rows for the parameters' gradients, any
// width: a thread owns eight columns and walks every parts-th row.
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
    float *p = a.part + (long long)blockIdx.y * 2 * a.cols;
    store8<Fp32>(p, c, a.cols, dg);
    store8<Fp32>(p + a.cols, c, a.cols, db);
}

// dgamma and dbeta: the partial sums in a fixed order.
__global__ __launch_bounds__(kLnThreads) void ln_bwd_reduce(const float *part, float *dgamma, float *dbeta, int cols,
                                                            int parts)
{
    const int c = blockIdx.x * kLnThreads + threadIdx.x;
    if (c >= cols)
        return;
    float g = 0.f, b = 0.f;
    for (int p = 0; p < parts; ++p) {
        g += part[(long long)p * 2 * cols + c];
        b += part[(long long)p * 2 * cols + cols + c];
    }
    dgamma[c] = g;
    dbeta[c] = b;
}

constexpr long long kMaxRows = 0x7fffffffLL;

// Workgroups for one a row: a launch holds fewer than 2^32 threads, so many
// rows are walked in strides of the grid.
unsigned ln_grid(long long rows) { return (unsigned)(rows < (1 << 22) ? rows : (1 << 22)); }

// Rows and columns each fit an int; all element offsets are 64-bit.
int ln_check(const void *x, long long ldx, long long rows, int cols, int dtype)
{
    if (rows < 0 || cols <= 0 || ldx < cols)
        return CONVIMG_ERR_SHAPE;
    if (!dtype_ok(dtype))
        return CONVIMG_ERR_DTYPE;
    if (rows > kMaxRows || cols > 0x7fffff00)
        return CONVIMG_ERR_RANGE;
    if (!x && rows > 0)
        return CONVIMG_ERR_NULL;
    return CONVIMG_OK;
}

template <typename X>
void ln_fwd_launch(const LnFwdArgs &a, int y_dtype, hipStream_t stream)
{
    const dim3 grid(ln_grid(a.rows));
    if (a.scales)
        hipLaunchKernelGGL((ln_fwd_wide<X, Mx4>), grid, dim3(kLnThreads), 0, stream, a);
    else
        with_dtype(y_dtype, [&](auto y) {
            hipLaunchKernelGGL((ln_fwd_wide<X, decltype(y)>), grid, dim3(kLnThreads), 0, stream, a);
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
    with_dtype(x_dtype, [&](auto x) { ln_fwd_launch<decltype(x)>(a, y_dtype, stream); });
    return hipGetLastError() == hipSuccess ? CONVIMG_OK : CONVIMG_ERR_LAUNCH;
}

constexpr int kLnMaxParts = 256;

int ln_parts(long long rows) { return (int)(rows < kLnMaxParts ? (rows > 0 ? rows : 1) : kLnMaxParts); }

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
    const int rc = ln_check(x, ldx, rows, cols, x_dtype);
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
    *bytes = (size_t)ln_parts(rows) * 2 * (size_t)cols * 4;
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
    const LnBwdArgs a = {dy,     x,     gamma, mean, rstd, dx,   (float *)ws, dgamma,
                         dbeta,  rows,  lddy,  ldx,  cols, dx_dtype, ln_parts(rows)};
    const int cgrid = (cols + 8 * kLnThreads - 1) / (8 * kLnThreads);
    with_dtype(dy_dtype, [&](auto d) {
        with_dtype(x_dtype, [&](auto t) {
            if (rows > 0)
                hipLaunchKernelGGL((ln_bwd_dx_wide<decltype(d), decltype(t)>), dim3(ln_grid(rows)),
                                   dim3(kLnThreads), 0, stream, a);
            if (dgamma)
                hipLaunchKernelGGL((ln_bwd_cols_wide<decltype(d), decltype(t)>), dim3(cgrid, a.parts),
                                   dim3(kLnThreads), 0, stream, a);
        });
    });
    if (dgamma)
        hipLaunchKernelGGL(ln_bwd_reduce, dim3((cols + kLnThreads - 1) / kLnThreads), dim3(kLnThreads), 0, stream,
                           a.part, dgamma, dbeta, cols, a.parts);
    return hipGetLastError() == hipSuccess ? CONVIMG_OK : CONVIMG_ERR_LAUNCH;
}

}  // extern "C"
