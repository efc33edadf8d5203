// mxfp4.hip -- microscaled 4-bit rows (MXFP4) and the linear layer on them.
//
// A block is 32 consecutive values of a row along the contracted axis.  With
// t the largest magnitude of a block, its scale is 2^(s - 127),
// s = clamp(floor(log2 t) - 2 + 127, 0, 254), and each value is stored as
// value / scale rounded to the nearest e2m1 number (0, .5, 1, 1.5, 2, 3, 4, 6
// with a sign; ties to the even code, saturating).
//
//   forward   y[m][n]  = sum_k Q(x)[m][k] Q(w)[n][k] + bias[n]
//   backward  dx[m][k] = sum_n Q(dy)[m][n] Q(w)[n][k]    blocks along n
//             dw[n][k] = sum_m Q(dy)[m][n] Q(x)[m][k]    blocks along m
//             db[n]    = sum_m dy[m][n]
//
// Products run on v_mfma_scale_f32_*_f8f6f4 with both operands e2m1 and one
// scale byte per lane and operand: a lane of the 32x32x64 form holds 32
// consecutive k of one row, which is one block, so blocks need no regrouping.
// Sums are fp32.
#include "mxfp4_gemm.hpp"

namespace convimg {

struct MxQuantArgs {
    const void *x;
    unsigned char *codes, *scales;
    long long ldx;
    int rows, cols;        // of x
    int lg;                // log2 of the threads a row
};

// Rows to MXFP4: a thread takes 8 columns, 4 neighbouring lanes a block.
template <typename T>
__global__ __launch_bounds__(kMxThreads) void mx_quantize_rows(MxQuantArgs a)
{
    const int tpr = 1 << a.lg;
    const long long row = (long long)blockIdx.x * (kMxThreads >> a.lg) + (threadIdx.x >> a.lg);
    if (row >= a.rows)
        return;
    const typename T::raw *x = (const typename T::raw *)a.x + row * a.ldx;
    const int kp = (a.cols + 31) & ~31;
    for (int c = (threadIdx.x & (tpr - 1)) * 8; c < kp; c += tpr * 8) {
        float v[8];
        load8<T>(x, c, a.cols, v);
        unsigned top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top = mx_top(top, v[e]);
        top = quad_max(top);
        const unsigned byte = mx_scale_byte(top);
        ((unsigned *)a.codes)[row * (kp / 8) + c / 8] = mx_encode8(v, mx_scale_value(byte));
        if ((c & 31) == 0) {
            unsigned char *s = a.scales + ((long long)(c >> 7) * a.rows + row) * 4;
            s[(c >> 5) & 3] = (unsigned char)byte;
            if (c + 32 == kp)      // bytes of blocks past the row's last one are 0
                for (int b = ((c >> 5) & 3) + 1; b < 4; ++b)
                    s[b] = 0;
        }
    }
}

// Columns to MXFP4 rows (blocks run down the columns of x): a thread takes
// 32 rows of one column.
template <typename T>
__global__ __launch_bounds__(kMxThreads) void mx_quantize_cols(MxQuantArgs a)
{
    const int col = blockIdx.x * kMxThreads + threadIdx.x;
    if (col >= a.cols)
        return;
    const int nb = mx_blocks(a.rows);
    for (int blk = blockIdx.y; blk < nb; blk += gridDim.y) {
        float v[32];
        unsigned top = 0;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            const int r = blk * 32 + e;
            v[e] = r < a.rows ? load1<T>((const typename T::raw *)a.x + r * a.ldx + col) : 0.f;
            top = mx_top(top, v[e]);
        }
        const unsigned byte = mx_scale_byte(top);
        const float scale = mx_scale_value(byte);
        u32v4_t q;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float w[8] = {v[8 * i], v[8 * i + 1], v[8 * i + 2], v[8 * i + 3],
                                v[8 * i + 4], v[8 * i + 5], v[8 * i + 6], v[8 * i + 7]};
            q[i] = mx_encode8(w, scale);
        }
        *(u32v4_t *)(a.codes + ((long long)col * nb + blk) * 16) = q;
        unsigned char *s = a.scales + ((long long)(blk >> 2) * a.cols + col) * 4;
        s[blk & 3] = (unsigned char)byte;
        if (blk + 1 == nb)
            for (int b = (blk & 3) + 1; b < 4; ++b)
                s[b] = 0;
    }
}

// MXFP4 rows to values: a thread takes 8 columns.
template <typename T>
__global__ __launch_bounds__(kMxThreads) void mx_dequantize_rows(const unsigned char *codes,
                                                                 const unsigned char *scales, void *out, int rows,
                                                                 int cols, int lg)
{
    const int tpr = 1 << lg;
    const long long row = (long long)blockIdx.x * (kMxThreads >> lg) + (threadIdx.x >> lg);
    if (row >= rows)
        return;
    const int kp = (cols + 31) & ~31;
    for (int c = (threadIdx.x & (tpr - 1)) * 8; c < cols; c += tpr * 8) {
        const unsigned byte = scales[((long long)(c >> 7) * rows + row) * 4 + ((c >> 5) & 3)];
        float v[8];
        mx_decode8(((const unsigned *)codes)[row * (kp / 8) + c / 8], mx_scale_value(byte), v);
        store8<T>((typename T::raw *)out + row * cols, c, cols, v);
    }
}

// Column sums of x in two steps: every parts-th row into part[p][cols], then
// the partial sums in a fixed order.
template <typename T>
__global__ __launch_bounds__(kMxThreads) void mx_colsum_part(const void *x, long long ldx, int rows, int cols,
                                                             float *part)
{
    const int c = blockIdx.x * kMxThreads + threadIdx.x;
    if (c >= cols)
        return;
    float s = 0.f;
    for (int r = blockIdx.y; r < rows; r += gridDim.y)
        s += load1<T>((const typename T::raw *)x + r * ldx + c);
    part[(long long)blockIdx.y * cols + c] = s;
}

__global__ __launch_bounds__(kMxThreads) void mx_colsum_reduce(const float *part, int parts, int cols, float *out)
{
    const int c = blockIdx.x * kMxThreads + threadIdx.x;
    if (c >= cols)
        return;
    float s = 0.f;
    for (int p = 0; p < parts; ++p)
        s += part[(long long)p * cols + c];
    out[c] = s;
}

// ---- host side -------------------------------------------------------------

struct MxOperand {
    const unsigned char *codes, *scales;
};

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Bytes of one packed operand in a workspace.
size_t packed_bytes(int rows, int cols)
{
    return align256(mx_code_bytes(rows, cols)) + align256(mx_scale_bytes(rows, cols));
}

// Threads a row (log2): enough for its columns, eight a thread, up to a
// workgroup; at least the four lanes of a block.
int row_lg(int cols)
{
    int lg = 2;
    while (lg < 8 && (8 << lg) < cols)
        ++lg;
    return lg;
}

unsigned row_grid(int rows, int lg) { return (unsigned)(((long long)rows + (kMxThreads >> lg) - 1) / (kMxThreads >> lg)); }

void quantize(const void *x, long long ldx, int rows, int cols, int dtype, bool transpose, unsigned char *codes,
              unsigned char *scales, hipStream_t stream)
{
    MxQuantArgs a = {x, codes, scales, ldx, rows, cols, row_lg(cols)};
    with_dtype(dtype, [&](auto t) {
        typedef decltype(t) T;
        if (!transpose) {
            hipLaunchKernelGGL(mx_quantize_rows<T>, dim3(row_grid(rows, a.lg)), dim3(kMxThreads), 0, stream, a);
        } else {
            const int nb = mx_blocks(rows);
            hipLaunchKernelGGL(mx_quantize_cols<T>, dim3((cols + kMxThreads - 1) / kMxThreads, nb < 65535 ? nb : 65535),
                               dim3(kMxThreads), 0, stream, a);
        }
    });
}

template <int BM, int BN, typename O>
void gemm_tiles(MxGemmArgs g, hipStream_t stream)
{
    g.tm = (g.M + BM - 1) / BM;
    g.tn = (g.N + BN - 1) / BN;
    const unsigned grid = (unsigned)(((long long)g.tm * g.tn + 7) / 8 * 8);
    hipLaunchKernelGGL((mx_gemm_tile<BM, BN, 4, O>), dim3(grid), dim3(kMxThreads), 0, stream, g);
}

void gemm(MxOperand a, MxOperand b, const float *bias, int M, int N, int K, int out_dtype, void *out,
          hipStream_t stream)
{
    const MxGemmArgs g = {a.codes, b.codes, a.scales, b.scales, bias, out, M, N, mx_blocks(K), 0, 0};
    auto tiles = [&](long long t) { return ((M + t - 1) / t) * ((N + t - 1) / t); };
    with_dtype(out_dtype, [&](auto o) {
        typedef decltype(o) O;
        if (tiles(256) >= 192)
            gemm_tiles<256, 256, O>(g, stream);
        else if (tiles(128) >= 192)
            gemm_tiles<128, 128, O>(g, stream);
        else
            gemm_tiles<64, 64, O>(g, stream);
    });
}

// Rows and columns of a packed operand: its codes stay below 2^31 bytes.
int mx_shape(long long rows, long long cols)
{
    if (rows < 0 || cols <= 0)
        return CONVIMG_ERR_SHAPE;
    if (rows > 0x7fffff00 || cols > 0x7fffff00 || mx_code_bytes(rows, (int)cols) >= 0x80000000u)
        return CONVIMG_ERR_RANGE;
    return CONVIMG_OK;
}

int launched() { return hipGetLastError() == hipSuccess ? CONVIMG_OK : CONVIMG_ERR_LAUNCH; }

constexpr int kMxSumParts = 128;
int sum_parts(int rows) { return rows < kMxSumParts ? (rows > 0 ? rows : 1) : kMxSumParts; }

bool misaligned(const void *p, unsigned n) { return ((uintptr_t)p & (n - 1)) != 0; }

// The four packed operands of the backward pass and the partial sums of db.
struct BwdLayout {
    size_t dy, wt, dyt, xt, part, total;
};

BwdLayout bwd_layout(int M, int N, int K)
{
    BwdLayout l;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += n;
        return here;
    };
    l.dy = take(packed_bytes(M, N));
    l.wt = take(packed_bytes(K, N));
    l.dyt = take(M > 0 ? packed_bytes(N, M) : 0);
    l.xt = take(M > 0 ? packed_bytes(K, M) : 0);
    l.part = take(align256((size_t)sum_parts(M) * N * 4));
    l.total = at;
    return l;
}

int bwd_shape(int M, int N, int K)
{
    int rc = mx_shape(M, N);
    if (rc == CONVIMG_OK)
        rc = mx_shape(M, K);
    if (rc == CONVIMG_OK)
        rc = mx_shape(N, K);
    if (rc == CONVIMG_OK)
        rc = mx_shape(K, N);
    if (rc == CONVIMG_OK && M > 0)
        rc = mx_shape(N, M);
    if (rc == CONVIMG_OK && M > 0)
        rc = mx_shape(K, M);
    return rc;
}

__global__ void mx_fill_zero(float *p, long long n)
{
    for (long long i = (long long)blockIdx.x * kMxThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kMxThreads)
        p[i] = 0.f;
}

void fill_zero(float *p, long long n, hipStream_t stream)
{
    const long long g = (n + kMxThreads - 1) / kMxThreads;
    hipLaunchKernelGGL(mx_fill_zero, dim3((unsigned)(g < 65536 ? g : 65536)), dim3(kMxThreads), 0, stream, p, n);
}

}  // namespace convimg

using namespace convimg;

extern "C" {

int mxfp4_bytes(long long rows, int cols, size_t *codes, size_t *scales)
{
    if (!codes || !scales)
        return CONVIMG_ERR_NULL;
    const int rc = mx_shape(rows, cols);
    if (rc != CONVIMG_OK)
        return rc;
    *codes = mx_code_bytes(rows, cols);
    *scales = mx_scale_bytes(rows, cols);
    return CONVIMG_OK;
}

int mxfp4_quantize(const void *x, long long ldx, int rows, int cols, int dtype, int transpose, void *codes,
                   void *scales, hipStream_t stream)
{
    if (rows < 0 || cols <= 0 || ldx < cols || (transpose && rows == 0))
        return CONVIMG_ERR_SHAPE;
    if (!dtype_ok(dtype))
        return CONVIMG_ERR_DTYPE;
    const int qr = transpose ? cols : rows, qc = transpose ? rows : cols;
    const int rc = mx_shape(qr, qc);
    if (rc != CONVIMG_OK)
        return rc;
    if (rows == 0)
        return CONVIMG_OK;
    if (!x || !codes || !scales)
        return CONVIMG_ERR_NULL;
    if (misaligned(codes, 16) || misaligned(scales, 4))
        return CONVIMG_ERR_ALIGN;
    const size_t nx = span_bytes(rows, ldx, cols, dtype), nc = mx_code_bytes(qr, qc), ns = mx_scale_bytes(qr, qc);
    if (row_overlaps(codes, nc, x, nx) || row_overlaps(scales, ns, x, nx) || row_overlaps(codes, nc, scales, ns))
        return CONVIMG_ERR_ALIAS;
    quantize(x, ldx, rows, cols, dtype, transpose != 0, (unsigned char *)codes, (unsigned char *)scales, stream);
    return launched();
}

int mxfp4_dequantize(const void *codes, const void *scales, int rows, int cols, int dtype, void *out,
                     hipStream_t stream)
{
    const int rc = mx_shape(rows, cols);
    if (rc != CONVIMG_OK)
        return rc;
    if (!dtype_ok(dtype))
        return CONVIMG_ERR_DTYPE;
    if (rows == 0)
        return CONVIMG_OK;
    if (!codes || !scales || !out)
        return CONVIMG_ERR_NULL;
    if (misaligned(codes, 16) || misaligned(scales, 4))
        return CONVIMG_ERR_ALIGN;
    const size_t no = span_bytes(rows, cols, cols, dtype);
    if (row_overlaps(out, no, codes, mx_code_bytes(rows, cols))
        || row_overlaps(out, no, scales, mx_scale_bytes(rows, cols)))
        return CONVIMG_ERR_ALIAS;
    const int lg = row_lg(cols);
    with_dtype(dtype, [&](auto t) {
        hipLaunchKernelGGL(mx_dequantize_rows<decltype(t)>, dim3(row_grid(rows, lg)), dim3(kMxThreads), 0, stream,
                           (const unsigned char *)codes, (const unsigned char *)scales, out, rows, cols, lg);
    });
    return launched();
}

int mxfp4_linear_workspace(int M, int N, int K, int x_dtype, size_t *bytes)
{
    if (!bytes)
        return CONVIMG_ERR_NULL;
    int rc = mx_shape(M, K);
    if (rc == CONVIMG_OK)
        rc = N <= 0 ? CONVIMG_ERR_SHAPE : mx_shape(N, K);
    if (rc != CONVIMG_OK)
        return rc;
    if (x_dtype != CONVIMG_MXFP4 && !dtype_ok(x_dtype))
        return CONVIMG_ERR_DTYPE;
    *bytes = x_dtype == CONVIMG_MXFP4 ? 0 : packed_bytes(M, K);
    return CONVIMG_OK;
}

int mxfp4_linear_fwd(const void *x, long long ldx, const void *x_scales, int x_dtype, const void *w_codes,
                     const void *w_scales, const float *bias, int M, int N, int K, int out_dtype, void *out, void *ws,
                     size_t ws_bytes, hipStream_t stream)
{
    size_t need = 0;
    const int rc = mxfp4_linear_workspace(M, N, K, x_dtype, &need);
    if (rc != CONVIMG_OK)
        return rc;
    if (!dtype_ok(out_dtype))
        return CONVIMG_ERR_DTYPE;
    const bool dense = x_dtype != CONVIMG_MXFP4;
    if (dense && ldx < K)
        return CONVIMG_ERR_SHAPE;
    if (M == 0)
        return CONVIMG_OK;
    if (!x || !w_codes || !w_scales || !out || (!dense && !x_scales) || (need > 0 && !ws))
        return CONVIMG_ERR_NULL;
    if (misaligned(w_codes, 16) || misaligned(w_scales, 4) || (need > 0 && misaligned(ws, 16))
        || (!dense && (misaligned(x, 16) || misaligned(x_scales, 4))))
        return CONVIMG_ERR_ALIGN;
    if (ws_bytes < need)
        return CONVIMG_ERR_WORKSPACE;
    const size_t no = span_bytes(M, N, N, out_dtype);
    const void *in[5] = {x, dense ? nullptr : x_scales, w_codes, w_scales, bias};
    const size_t nin[5] = {dense ? span_bytes(M, ldx, K, x_dtype) : mx_code_bytes(M, K), mx_scale_bytes(M, K),
                           mx_code_bytes(N, K), mx_scale_bytes(N, K), (size_t)N * 4};
    for (int i = 0; i < 5; ++i)
        if (row_overlaps(out, no, in[i], nin[i]) || row_overlaps(ws, need, in[i], nin[i]))
            return CONVIMG_ERR_ALIAS;
    if (row_overlaps(out, no, ws, need))
        return CONVIMG_ERR_ALIAS;
    MxOperand a = {(const unsigned char *)x, (const unsigned char *)x_scales};
    const MxOperand b = {(const unsigned char *)w_codes, (const unsigned char *)w_scales};
    if (dense) {
        unsigned char *c = (unsigned char *)ws, *s = c + align256(mx_code_bytes(M, K));
        quantize(x, ldx, M, K, x_dtype, false, c, s, stream);
        a = {c, s};
    }
    gemm(a, b, bias, M, N, K, out_dtype, out, stream);
    return launched();
}

int mxfp4_linear_bwd_workspace(int M, int N, int K, size_t *bytes)
{
    if (!bytes)
        return CONVIMG_ERR_NULL;
    const int rc = bwd_shape(M, N, K);
    if (rc != CONVIMG_OK)
        return rc;
    *bytes = bwd_layout(M, N, K).total;
    return CONVIMG_OK;
}

int mxfp4_linear_bwd(const void *dy, long long lddy, int dy_dtype, const void *x, long long ldx, const void *w,
                     long long ldw, int dtype, int M, int N, int K, int dx_dtype, void *dx, float *dw, float *db,
                     void *ws, size_t ws_bytes, hipStream_t stream)
{
    const int rc = bwd_shape(M, N, K);
    if (rc != CONVIMG_OK)
        return rc;
    if (lddy < N || ldx < K || ldw < K)
        return CONVIMG_ERR_SHAPE;
    if (!dtype_ok(dy_dtype) || !dtype_ok(dtype) || !dtype_ok(dx_dtype))
        return CONVIMG_ERR_DTYPE;
    if ((M > 0 && (!dy || !x || !dx)) || !w || !dw || !ws)
        return CONVIMG_ERR_NULL;
    if (misaligned(ws, 16))
        return CONVIMG_ERR_ALIGN;
    const BwdLayout l = bwd_layout(M, N, K);
    if (ws_bytes < l.total)
        return CONVIMG_ERR_WORKSPACE;
    const void *in[3] = {dy, x, w};
    const size_t nin[3] = {span_bytes(M, lddy, N, dy_dtype), span_bytes(M, ldx, K, dtype), span_bytes(N, ldw, K, dtype)};
    const void *out[4] = {dx, dw, db, ws};
    const size_t nout[4] = {span_bytes(M, K, K, dx_dtype), (size_t)N * K * 4, (size_t)N * 4, l.total};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 3; ++j)
            if (row_overlaps(out[i], nout[i], in[j], nin[j]))
                return CONVIMG_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (row_overlaps(out[i], nout[i], out[j], nout[j]))
                return CONVIMG_ERR_ALIAS;
    }
    if (M == 0) {      // no pixel: the parameters' gradients are 0
        fill_zero(dw, (long long)N * K, stream);
        if (db)
            fill_zero(db, N, stream);
        return launched();
    }
    unsigned char *base = (unsigned char *)ws;
    auto operand = [&](size_t at, int rows, int cols) {
        return MxOperand{base + at, base + at + align256(mx_code_bytes(rows, cols))};
    };
    auto pack = [&](const void *p, long long ld, int rows, int cols, int t, bool tr, MxOperand o) {
        quantize(p, ld, rows, cols, t, tr, (unsigned char *)o.codes, (unsigned char *)o.scales, stream);
    };
    const MxOperand qdy = operand(l.dy, M, N), qwt = operand(l.wt, K, N), qdyt = operand(l.dyt, N, M),
                    qxt = operand(l.xt, K, M);
    pack(dy, lddy, M, N, dy_dtype, false, qdy);
    pack(w, ldw, N, K, dtype, true, qwt);
    pack(dy, lddy, M, N, dy_dtype, true, qdyt);
    pack(x, ldx, M, K, dtype, true, qxt);
    gemm(qdy, qwt, nullptr, M, K, N, dx_dtype, dx, stream);
    gemm(qdyt, qxt, nullptr, N, K, M, CONVIMG_FP32, dw, stream);
    if (db) {
        float *part = (float *)(base + l.part);
        const dim3 grid((N + kMxThreads - 1) / kMxThreads, sum_parts(M));
        with_dtype(dy_dtype, [&](auto t) {
            hipLaunchKernelGGL(mx_colsum_part<decltype(t)>, grid, dim3(kMxThreads), 0, stream, dy, lddy, M, N, part);
        });
        hipLaunchKernelGGL(mx_colsum_reduce, dim3(grid.x), dim3(kMxThreads), 0, stream, part, sum_parts(M), N, db);
    }
    return launched();
}

}  // extern "C"
