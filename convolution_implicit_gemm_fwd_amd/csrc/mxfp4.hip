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
#include <type_traits>

#include "mxfp4_plan.hpp"

namespace convimg {

// ---- host side -------------------------------------------------------------

void quantize(const void *x, long long ldx, int rows, int cols, int dtype, unsigned char *codes,
              unsigned char *scales, hipStream_t stream)
{
    const MxQuantArgs a = {x, codes, scales, ldx, rows, cols, row_lg(cols)};
    with_dtype(dtype, [&](auto t) {
        hipLaunchKernelGGL(mx_quantize_rows<decltype(t)>, dim3(eights(row_grid(rows, a.lg))), dim3(kMxThreads), 0, stream, a);
    });
}

void quantize_cols(const void *x, long long ldx, int rows, int cols, int dtype, unsigned char *codes,
                   unsigned char *scales, hipStream_t stream)
{
    const MxTileArgs a = {x, nullptr, ldx, rows, cols, codes, scales, nullptr, nullptr, nullptr};
    const long long tiles = mx_tiles(rows, cols);
    // (a launch holds fewer than 2^32 threads: 2^30 rows of one column are 2^23 tiles)
    constexpr long long kStep = 1 << 21;
    with_dtype(dtype, [&](auto t) {
        for (long long first = 0; first < tiles; first += kStep) {
            const long long end = first + kStep < tiles ? first + kStep : tiles;
            hipLaunchKernelGGL(mx_quantize_cols<decltype(t)>, dim3(eights(end - first)), dim3(kMxTileThreads), 0, stream,
                               a, (unsigned)first, (unsigned)end);
        }
    });
}

void gemm(MxGemmArgs g, int out_dtype, hipStream_t stream)
{
    with_dtype(out_dtype, [&](auto o) {
        with_shape(shape_of(tiles_of(g.M, g.N), g.kb), [&](auto shape) {
            typedef decltype(shape) S;
            const unsigned grid = gemm_grid(g, S::BM, S::BN);
            hipLaunchKernelGGL((mx_gemm_tile<S, decltype(o)>), dim3(grid), dim3(S::threads), 0, stream, g);
        });
    });
}

void gemm_few(const MxFewArgs &g, int x_dtype, int out_dtype, hipStream_t stream)
{
    // a wave for every pair of scale dwords, up to eight
    const int pairs = (g.kb + 7) / 8, waves = pairs < kMxFewWaves ? pairs : kMxFewWaves;
    with_dtype(x_dtype, [&](auto x) {
        with_dtype(out_dtype, [&](auto o) {
            hipLaunchKernelGGL((mx_gemm_few<decltype(x), decltype(o)>), dim3((g.N + 15) / 16), dim3(waves * 64), 0,
                               stream, g, MxNoAdapters{});
        });
    });
}

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
    l.part = take(align256((size_t)((M + kMxTile - 1) / kMxTile) * N * 4));
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

// The gradient of the linear layer, x dense or (kept) in 8 bits with scale
// bytes xs.
int linear_bwd(const void *dy, long long lddy, int dy_dtype, const void *x, const void *xs, long long ldx,
               const void *w, long long ldw, int dtype, int M, int N, int K, int dx_dtype, void *dx, float *dw,
               float *db, void *ws, size_t ws_bytes, hipStream_t stream, bool kept)
{
    const int rc = bwd_shape(M, N, K);
    if (rc != CONVIMG_OK)
        return rc;
    if (lddy < N || ldx < K || ldw < K)
        return CONVIMG_ERR_SHAPE;
    if (!dtype_ok(dy_dtype) || !dtype_ok(dtype) || !dtype_ok(dx_dtype))
        return CONVIMG_ERR_DTYPE;
    if ((M > 0 && (!dy || !x || !dx || (kept && !xs))) || !w || !dw || !ws)
        return CONVIMG_ERR_NULL;
    if (misaligned(ws, 16) || (kept && (misaligned(x, 16) || misaligned(xs, 4))))
        return CONVIMG_ERR_ALIGN;
    const BwdLayout l = bwd_layout(M, N, K);
    if (ws_bytes < l.total)
        return CONVIMG_ERR_WORKSPACE;
    const void *in[4] = {dy, x, w, xs};
    const size_t nin[4] = {span_bytes(M, lddy, N, dy_dtype), kept ? mxi_code_bytes(M, K) : span_bytes(M, ldx, K, dtype),
                           span_bytes(N, ldw, K, dtype), kept ? mxi_scale_bytes(M, K) : 0};
    const void *out[4] = {dx, dw, db, ws};
    const size_t nout[4] = {span_bytes(M, K, K, dx_dtype), (size_t)N * K * 4, (size_t)N * 4, l.total};
    if (any_overlap(out, nout, 4, in, nin, 4))
        return CONVIMG_ERR_ALIAS;
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
    const MxOperand qdy = operand(l.dy, M, N), qwt = operand(l.wt, K, N), qdyt = operand(l.dyt, N, M),
                    qxt = operand(l.xt, K, M);
    float *part = (float *)(base + l.part);
    auto tiles = [](const void *p, const void *ps, long long ld, int rows, int cols, MxOperand down, MxOperand along,
                    float *sums) {
        return MxTileArgs{p,
                          (const unsigned char *)ps,
                          ld,
                          rows,
                          cols,
                          (unsigned char *)down.codes,
                          (unsigned char *)down.scales,
                          (unsigned char *)along.codes,
                          (unsigned char *)along.scales,
                          sums};
    };
    const long long t_dy = mx_tiles(M, N), t_w = mx_tiles(N, K), t_x = mx_tiles(M, K);
    const MxTileArgs a_dy = tiles(dy, nullptr, lddy, M, N, qdyt, qdy, part),
                     a_w = tiles(w, nullptr, ldw, N, K, qwt, {}, nullptr),
                     a_x = tiles(x, xs, ldx, M, K, qxt, {}, nullptr);
    with_dtype(dy_dtype, [&](auto d) {
        with_dtype(dtype, [&](auto t) {
            auto launch = [&](auto k) {
                hipLaunchKernelGGL((mx_quantize_bwd<decltype(d), decltype(t), decltype(k)::value>),
                                   dim3(eights(t_dy) + eights(t_w) + eights(t_x)), dim3(kMxTileThreads), 0, stream, a_dy,
                                   a_w, a_x, (unsigned)t_dy, (unsigned)t_w, (unsigned)t_x);
            };
            if (kept)
                launch(std::true_type{});
            else
                launch(std::false_type{});
        });
    });
    MxGemmArgs g_dx = gemm_args(qdy, qwt, nullptr, M, K, N, dx), g_dw = gemm_args(qdyt, qxt, nullptr, N, K, M, dw);
    const MxSumArgs sum = {part, db, (M + kMxTile - 1) / kMxTile, N};
    // One launch for both products where they want tiles of like size; else
    // the smaller one's few large tiles would be the last to end.
    Shape s_dw = shape_of(tiles_of(N, K), g_dw.kb);
    const Shape s_dx = shape_of(tiles_of(M, K), g_dx.kb);
    const int apart = shape_level(s_dw) - shape_level(s_dx);
    const bool both = apart < 2 && apart > -2;
    if (both)
        s_dw = shape_of([&](int bm, int bn) { return tile_count(M, K, bm, bn) + tile_count(N, K, bm, bn); },
                        M > N ? g_dw.kb : g_dx.kb);
    with_dtype(dx_dtype, [&](auto o) {
        with_shape(s_dw, [&](auto shape) {
            typedef decltype(shape) S;
            const unsigned n_dx = both ? gemm_grid(g_dx, S::BM, S::BN) : 0, n_dw = gemm_grid(g_dw, S::BM, S::BN),
                           n_db = db ? (N + 63) / 64 : 0;
            hipLaunchKernelGGL((mx_gemm_bwd<S, decltype(o)>), dim3(n_dw + n_dx + n_db), dim3(S::threads), 0, stream,
                               g_dw, g_dx, sum, n_dw, n_dx);
        });
    });
    if (!both)
        gemm(g_dx, dx_dtype, stream);
    return launched();
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
    if (transpose)
        quantize_cols(x, ldx, rows, cols, dtype, (unsigned char *)codes, (unsigned char *)scales, stream);
    else
        quantize(x, ldx, rows, cols, dtype, (unsigned char *)codes, (unsigned char *)scales, stream);
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
    *bytes = x_dtype == CONVIMG_MXFP4 || few_dense(M, K) ? 0 : packed_bytes(M, K);
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
    if (dense && need == 0) {
        gemm_few({x, b.codes, b.scales, bias, out, ldx, M, N, K, mx_blocks(K)}, x_dtype, out_dtype, stream);
        return launched();
    }
    if (dense) {
        unsigned char *c = (unsigned char *)ws, *s = c + align256(mx_code_bytes(M, K));
        quantize(x, ldx, M, K, x_dtype, c, s, stream);
        a = {c, s};
    }
    gemm(gemm_args(a, b, bias, M, N, K, out), out_dtype, stream);
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
    return linear_bwd(dy, lddy, dy_dtype, x, nullptr, ldx, w, ldw, dtype, M, N, K, dx_dtype, dx, dw, db, ws, ws_bytes,
                      stream, false);
}

int mxfp4_linear_bwd_mxint8(const void *dy, long long lddy, int dy_dtype, const void *x_codes, const void *x_scales,
                            const void *w, long long ldw, int w_dtype, int M, int N, int K, int dx_dtype, void *dx,
                            float *dw, float *db, void *ws, size_t ws_bytes, hipStream_t stream)
{
    return linear_bwd(dy, lddy, dy_dtype, x_codes, x_scales, K, w, ldw, w_dtype, M, N, K, dx_dtype, dx, dw, db, ws,
                      ws_bytes, stream, true);
}

}  // extern "C"
