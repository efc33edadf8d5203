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

#include "mxfp4_few.hpp"

namespace convimg {

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

unsigned eights(long long n) { return (unsigned)((n + 7) / 8 * 8); }

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
    const MxTileArgs a = {x, ldx, rows, cols, codes, scales, nullptr, nullptr, nullptr};
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

long long tile_count(int M, int N, int bm, int bn) { return (long long)((M + bm - 1) / bm) * ((N + bn - 1) / bn); }

auto tiles_of(int M, int N)
{
    return [=](int bm, int bn) { return tile_count(M, N, bm, bn); };
}

// The shape for a launch that has count(BM, BN) tiles and kb blocks along K: the largest tile that still gives most of the 256 CUs one.
// Measured on both sides of each bound (M x N x K, us):
//   256 x 256 from 144 tiles: 3000^3 28.9 (144 tiles) against 31.7 in 128 x
//     128; 2048x4096x4096 (128 tiles) 31.8 against 23.9.
//   128 x 128 from 192: 1024x4096x4096 (256) 16.7 against 20.6 in 128 x 64.
//   128 x 64, two groups of waves, from 192: 512x4096x4096 (256) 11.2 against
//     15.1 in 128 x 128 and 12.8 in 64 x 64; 256x4096x4096 (128) 10.6 against 8.6.
//   64 x 64 from 192, and where K is at most 1024: 512^3 3.4 against 4.0 in 32 x 32;
//     K tiles of 128, which hide more of the latency that such launches consist
//     of than whole cache lines save (37x8000x4096 8.0, against 10.8 us in tiles of 256).
//   64 x 32, four groups, from 192: 128x4096x4096 (256) 7.0 against 7.7 in 32 x 32.
//   else 32 x 32: 64x4096x4096 6.3 against 6.9 in 64 x 32.
//   Where K is at most 256 (512 in very many tiles) the output is the work:
//     128 x 128 with two short stages, of which a CU holds three workgroups, so
//     that one stores while others load: 8192x8192x256 30.5 us against 38.3 in
//     256 x 256, x512 38.1 against 42.1, x1024 59.9 against 55.6; 3136x2048x512
//     (400 tiles) 8.7 against 8.3 in the longer stages.
//   Where K is at most 2048, the last round of 256 x 256 tiles would leave more
//     than 15 % of all rounds idle and there are 1024 tiles of 128 x 128, those,
//     which overlap anyway: 7000x7000x1000 47.5 us against 61.0, 6000x6000x2000
//     62.4 against 65.6, 4100x4100 (1089 tiles) x1000 21.5 against 26.4 and x2000
//     34.9 against 40.9; without that rest 8192x4096x2048 48.5 against 48.0.
//     With fewer tiles the larger ones are one round, and either may win:
//     3500x3500 (784) x1000 16.7 against 19.2 and x2000 26.1 against 26.8,
//     3328x3328 (676) 14.3 against 14.4 and 23.7 against 22.0.
enum Shape { k256, k128, k128Short, k128x64, k64, k64x32, k32 };

template <typename C>
Shape shape_of(C &&count, int kb)
{
    const long long n = count(128, 128);
    if (n >= 192 && (kb <= 8 || (kb <= 16 && n >= 2048)))
        return k128Short;
    const long long big = count(256, 256), rounds = (big + 255) / 256;
    if (big >= 144 && !(kb <= 64 && n >= 1024 && big * 100 < rounds * 256 * 85))
        return k256;
    if (n >= 192)
        return k128;
    if (count(128, 64) >= 192 && kb > 32)
        return k128x64;
    if (count(64, 64) >= 192 || kb <= 32)
        return k64;
    return count(64, 32) >= 192 ? k64x32 : k32;
}

// Steps in tile size (the two 128 x 128 shapes are one).
int shape_level(Shape s) { return s <= k128 ? s : s - 1; }

template <typename F>
void with_shape(Shape shape, F &&f)
{
    switch (shape) {
    case k256: f(GemmShape<256, 256, 2, 2, 256, 2, 1>{}); break;
    case k128: f(GemmShape<128, 128, 2, 2, 256, 2, 1>{}); break;
    case k128Short: f(GemmShape<128, 128, 2, 2, 128, 2, 1>{}); break;
    case k128x64: f(GemmShape<128, 64, 2, 2, 256, 2, 2>{}); break;
    case k64: f(GemmShape<64, 64, 2, 2, 128, 4, 1>{}); break;
    case k64x32: f(GemmShape<64, 32, 2, 1, 256, 2, 4>{}); break;
    case k32: f(GemmShape<32, 32, 1, 1, 256, 2, 4>{}); break;
    }
}

MxGemmArgs gemm_args(MxOperand a, MxOperand b, const float *bias, int M, int N, int K, void *out)
{
    return {a.codes, b.codes, a.scales, b.scales, bias, out, M, N, mx_blocks(K), 0, 0};
}

unsigned gemm_grid(MxGemmArgs &g, int bm, int bn)
{
    g.tm = (g.M + bm - 1) / bm;
    g.tn = (g.N + bn - 1) / bn;
    return eights((long long)g.tm * g.tn);
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

// Dense rows that the product's workgroups quantise for themselves: one
// launch in place of two, while that costs each workgroup little.  In one
// launch against two (us): 4096 -> 4096 3.9 against 7.4 for one row, 5.3 against
// 7.5 for four; 4096 -> 8000 6.2 against 9.5 and 7.6 against 9.6; 8192 -> 8192
// 9.8 against 13.9 and, at both bounds, 13.5 against 13.9; 16384 -> 4096 11.6
// against 19.0 for two rows.  Past the bounds, with LDS for 16 rows: 4096 -> 8000
// 10.6 against 9.7 for five rows and 14.0 against 9.6 for eight, 4096 -> 4096
// 5.9 against 7.7, 7.3 against 7.8 and, for 16, 10.9 against 8.0; 8192 -> 8192
// 18.8 against 13.9 for five; 16384 -> 4096 15.6 against 18.8 for four.
bool few_dense(int M, int K) { return M <= kMxFewM && (long long)M * K <= kMxFewSize; }

void gemm_few(const MxFewArgs &g, int x_dtype, int out_dtype, hipStream_t stream)
{
    // a wave for every pair of scale dwords, up to eight
    const int pairs = (g.kb + 7) / 8, waves = pairs < kMxFewWaves ? pairs : kMxFewWaves;
    with_dtype(x_dtype, [&](auto x) {
        with_dtype(out_dtype, [&](auto o) {
            hipLaunchKernelGGL((mx_gemm_few<decltype(x), decltype(o)>), dim3((g.N + 15) / 16), dim3(waves * 64), 0,
                               stream, g);
        });
    });
}

int launched() { return hipGetLastError() == hipSuccess ? CONVIMG_OK : CONVIMG_ERR_LAUNCH; }

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
    const MxOperand qdy = operand(l.dy, M, N), qwt = operand(l.wt, K, N), qdyt = operand(l.dyt, N, M),
                    qxt = operand(l.xt, K, M);
    float *part = (float *)(base + l.part);
    auto tiles = [](const void *p, long long ld, int rows, int cols, MxOperand down, MxOperand along, float *sums) {
        return MxTileArgs{p,
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
    const MxTileArgs a_dy = tiles(dy, lddy, M, N, qdyt, qdy, part), a_w = tiles(w, ldw, N, K, qwt, {}, nullptr),
                     a_x = tiles(x, ldx, M, K, qxt, {}, nullptr);
    with_dtype(dy_dtype, [&](auto d) {
        with_dtype(dtype, [&](auto t) {
            hipLaunchKernelGGL((mx_quantize_bwd<decltype(d), decltype(t)>), dim3(eights(t_dy) + eights(t_w) + eights(t_x)),
                               dim3(kMxTileThreads), 0, stream, a_dy, a_w, a_x, (unsigned)t_dy, (unsigned)t_w,
                               (unsigned)t_x);
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

}  // extern "C"
