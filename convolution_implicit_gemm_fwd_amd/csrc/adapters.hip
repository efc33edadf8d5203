// adapters.hip -- low-rank adapters of many requests beside the linear layer
// on 4-bit rows: entry points, and the products with the adapters' second half
// (adapter_expand.hpp) inside.
//
//   h[m]   = down_g x[m],  g = ids[m]              a pass over x that quantises it, too
//   out[m] = Q(x[m]) W^T + bias + scale_g h[m] up_g     the product
//
// Backward, with t[m] = up_g dy[m], the same two steps with down and up
// exchanged, and the adapters' gradients from t and x, h and dy.
#include "adapter.hpp"

namespace convimg {

// adapter_grads_*.hip, by the type of dy
void adapter_grads_bf16(const AdGradArgs &up, const AdGradArgs &down, int x_dtype, hipStream_t stream);
void adapter_grads_fp16(const AdGradArgs &up, const AdGradArgs &down, int x_dtype, hipStream_t stream);
void adapter_grads_fp32(const AdGradArgs &up, const AdGradArgs &down, int x_dtype, hipStream_t stream);

// adapter_products_*.hip, by the type of the adapters
void gemm_adapters_bf16(const MxGemmArgs &g, const MxAdapterArgs &ad, int out_dtype, hipStream_t stream);
void few_adapters_bf16(const MxFewArgs &g, const MxAdapterArgs &ad, int x_dtype, int out_dtype, hipStream_t stream);
void gemm_adapters_fp16(const MxGemmArgs &g, const MxAdapterArgs &ad, int out_dtype, hipStream_t stream);
void few_adapters_fp16(const MxFewArgs &g, const MxAdapterArgs &ad, int x_dtype, int out_dtype, hipStream_t stream);
void gemm_adapters_fp32(const MxGemmArgs &g, const MxAdapterArgs &ad, int out_dtype, hipStream_t stream);
void few_adapters_fp32(const MxFewArgs &g, const MxAdapterArgs &ad, int x_dtype, int out_dtype, hipStream_t stream);

void gemm_adapters(const MxGemmArgs &g, const MxAdapterArgs &ad, int out_dtype, hipStream_t stream)
{
    auto f = ad.dtype == CONVIMG_BF16 ? gemm_adapters_bf16 : ad.dtype == CONVIMG_FP16 ? gemm_adapters_fp16 : gemm_adapters_fp32;
    f(g, ad, out_dtype, stream);
}

void few_adapters(const MxFewArgs &g, const MxAdapterArgs &ad, int x_dtype, int out_dtype, hipStream_t stream)
{
    auto f = ad.dtype == CONVIMG_BF16 ? few_adapters_bf16 : ad.dtype == CONVIMG_FP16 ? few_adapters_fp16 : few_adapters_fp32;
    f(g, ad, x_dtype, out_dtype, stream);
}

constexpr int kMaxRank = 4096;

// Columns of an adapter at most: 16 rows of it stay below 2^31 bytes.
constexpr int kMaxAdapterCols = (1 << 25) - 1;
// Rows: a launch with a workgroup of 512 threads for 16 of them holds fewer than 2^32 threads.
constexpr int kMaxAdapterRows = (1 << 26) - 1;

int adapters_shape(int M, int N, int K, int adapters, int rank)
{
    int rc = mx_shape(M, K);
    if (rc == CONVIMG_OK)
        rc = N <= 0 ? CONVIMG_ERR_SHAPE : mx_shape(N, K);
    if (rc == CONVIMG_OK)
        rc = rank <= 0 || adapters <= 0 ? CONVIMG_ERR_SHAPE
             : rank > kMaxRank || N > kMaxAdapterCols || K > kMaxAdapterCols || M > kMaxAdapterRows ? CONVIMG_ERR_RANGE
                                                                                                   : CONVIMG_OK;
    return rc;
}

// Workspace of the forward call: x's packed rows, h, its terms and the sorted
// order.
struct AdFwdLayout {
    size_t h, terms, order, total;
    AdPlan plan;
};

size_t ad_h_bytes(int M, int rank) { return align256((size_t)M * adapter_ranks(rank) * 4); }
size_t ad_term_bytes(int M, int rank) { return align256((size_t)M * (adapter_ranks(rank) / 16) * kAdTermBytes); }

AdFwdLayout ad_fwd_layout(int M, int K, int G, int rank)
{
    AdFwdLayout l;
    const bool few = few_dense(M, K);      // (its product takes the rows as they are)
    l.plan = adapter_plan(M, G);
    l.h = few ? 0 : packed_bytes(M, K);
    l.terms = l.h + ad_h_bytes(M, rank);
    l.order = l.terms + (few ? 0 : ad_term_bytes(M, rank));
    l.total = l.order + (l.plan.sorted ? (size_t)M * 12 + ((size_t)G + 1) * 4 : 0);
    return l;
}

int grad_tiles(int C) { return (int)((C + 127LL) / 128); }
int grad_chunks_of_ranks(int r) { return (r + 63) / 64; }

// Sorted rows a chunk of the gradients: so many that there are about 512
// workgroups, in runs of 32 rows.  (With 1024 the 8192 rows above 4096 columns
// take 35 us instead of 33.6, and the sums over the chunks 6.6 instead of 6.3.)
int adapter_grad_per(int M, int C, int r)
{
    const long long tiles = (long long)grad_tiles(C) * grad_chunks_of_ranks(r), chunks = tiles < 512 ? 512 / tiles : 1,
                    per = (M + chunks - 1) / chunks;
    return (int)((per + 31) / 32 * 32 < 32 ? 32 : (per + 31) / 32 * 32);
}

struct AdBwdLayout {
    size_t dy, t, terms, part_down, part_up, order, start, nan, total;
    int per_down, per_up;
};

int ad_chunks(int M, int per) { return (int)((M + (long long)per - 1) / per); }

AdBwdLayout ad_bwd_layout(int M, int N, int K, int G, int rank)
{
    AdBwdLayout l;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += align256(n);
        return here;
    };
    l.per_down = adapter_grad_per(M, K, rank);
    l.per_up = adapter_grad_per(M, N, rank);
    l.dy = take(packed_bytes(M, N));
    l.t = take(ad_h_bytes(M, rank));
    l.terms = take(ad_term_bytes(M, rank));
    l.part_down = take((size_t)ad_chunks(M, l.per_down) * 2 * rank * K * 4);
    l.part_up = take((size_t)ad_chunks(M, l.per_up) * 2 * rank * N * 4);
    l.order = take((size_t)M * 12);
    l.start = take(((size_t)G + 1) * 4);
    l.nan = take(4);
    l.total = at;
    return l;
}

int ad_bwd_shape(int M, int N, int K, int adapters, int rank)
{
    const int rc = adapters_shape(M, K, N, adapters, rank);      // dy's rows and wt's
    if (rc != CONVIMG_OK)
        return rc;
    // (the gradients' launch: a workgroup of 256 threads for 128 columns and 64 ranks)
    if (((long long)grad_tiles(N) + grad_tiles(K)) * grad_chunks_of_ranks(rank) > (1 << 22))
        return CONVIMG_ERR_RANGE;
    return mx_shape(M, K);
}

}  // namespace convimg

using namespace convimg;

extern "C" {

int mxfp4_linear_adapters_workspace(int M, int N, int K, int adapters, int rank, int x_dtype, size_t *bytes)
{
    if (!bytes)
        return CONVIMG_ERR_NULL;
    const int rc = adapters_shape(M, N, K, adapters, rank);
    if (rc != CONVIMG_OK)
        return rc;
    if (!dtype_ok(x_dtype))
        return CONVIMG_ERR_DTYPE;
    *bytes = ad_fwd_layout(M, K, adapters, rank).total;
    return CONVIMG_OK;
}

int mxfp4_linear_adapters_fwd(const void *x, long long ldx, int x_dtype, const void *w_codes, const void *w_scales,
                              const float *bias, const void *down, const void *up, const float *scale, const int *ids,
                              int adapters, int rank, int a_dtype, int M, int N, int K, int out_dtype, void *out,
                              float *h, void *x_codes, void *x_scales, void *ws, size_t ws_bytes, hipStream_t stream)
{
    size_t need = 0;
    const int rc = mxfp4_linear_adapters_workspace(M, N, K, adapters, rank, x_dtype, &need);
    if (rc != CONVIMG_OK)
        return rc;
    if (!dtype_ok(out_dtype) || !dtype_ok(a_dtype))
        return CONVIMG_ERR_DTYPE;
    if (ldx < K)
        return CONVIMG_ERR_SHAPE;
    if (M == 0)
        return CONVIMG_OK;
    if (!x || !w_codes || !w_scales || !down || !up || !scale || !ids || !out || !ws || (!x_codes) != (!x_scales))
        return CONVIMG_ERR_NULL;
    if (misaligned(w_codes, 16) || misaligned(w_scales, 4) || misaligned(ws, 16) || misaligned(x_codes, 16)
        || misaligned(x_scales, 4))
        return CONVIMG_ERR_ALIGN;
    if (ws_bytes < need)
        return CONVIMG_ERR_WORKSPACE;
    const size_t na = (size_t)adapters * rank * dtype_bytes(a_dtype);
    const void *in[8] = {x, w_codes, w_scales, bias, down, up, scale, ids}, *outs[5] = {out, h, x_codes, x_scales, ws};
    const size_t nin[8] = {span_bytes(M, ldx, K, x_dtype), mx_code_bytes(N, K), mx_scale_bytes(N, K), (size_t)N * 4, na * K,
                           na * N, (size_t)adapters * 4, (size_t)M * 4},
                 nout[5] = {span_bytes(M, N, N, out_dtype), (size_t)M * rank * 4, mxi_code_bytes(M, K),
                            mxi_scale_bytes(M, K), need};
    if (any_overlap(outs, nout, 5, in, nin, 8))
        return CONVIMG_ERR_ALIAS;
    const AdFwdLayout l = ad_fwd_layout(M, K, adapters, rank);
    unsigned char *base = (unsigned char *)ws, *codes = l.h ? base : nullptr,
                  *scales = codes ? codes + align256(mx_code_bytes(M, K)) : nullptr,
                  *terms = codes ? base + l.terms : nullptr;
    int *order = l.plan.sorted ? (int *)(base + l.order) : nullptr;
    const int *key = order ? order + 2LL * M : ids;
    int *start = order ? order + 3LL * M : nullptr;
    float *hh = (float *)(base + l.h);
    if (order)
        adapter_sort(ids, M, adapters, order, order + 2LL * M, start, nullptr, stream);
    const AdShrinkArgs s = {x, down, scale, key, order, start, hh, terms, h, codes, scales, (unsigned char *)x_codes,
                            (unsigned char *)x_scales, ldx, M, K, adapters, rank};
    adapter_shrink(s, l.plan, x_dtype, a_dtype, stream);
    const MxAdapterArgs ad = {terms, hh, up, scale, key, order, adapters, rank, a_dtype};
    const MxOperand b = {(const unsigned char *)w_codes, (const unsigned char *)w_scales};
    if (!codes)
        few_adapters({x, b.codes, b.scales, bias, out, ldx, M, N, K, mx_blocks(K)}, ad, x_dtype, out_dtype, stream);
    else
        gemm_adapters(gemm_args({codes, scales}, b, bias, M, N, K, out), ad, out_dtype, stream);
    return launched();
}

int mxfp4_linear_adapters_bwd_workspace(int M, int N, int K, int adapters, int rank, size_t *bytes)
{
    if (!bytes)
        return CONVIMG_ERR_NULL;
    const int rc = ad_bwd_shape(M, N, K, adapters, rank);
    if (rc != CONVIMG_OK)
        return rc;
    *bytes = ad_bwd_layout(M, N, K, adapters, rank).total;
    return CONVIMG_OK;
}

int mxfp4_linear_adapters_bwd(const void *dy, long long lddy, int dy_dtype, const void *x, long long ldx,
                              const void *x_scales, int x_dtype, const void *wt_codes, const void *wt_scales,
                              const void *down, const void *up, const float *scale, const int *ids, int adapters,
                              int rank, int a_dtype, const float *h, int M, int N, int K, int dx_dtype, void *dx,
                              float *ddown, float *dup, void *ws, size_t ws_bytes, hipStream_t stream)
{
    const int rc = ad_bwd_shape(M, N, K, adapters, rank);
    if (rc != CONVIMG_OK)
        return rc;
    const bool kept = x_dtype == CONVIMG_MXINT8;
    if (!dtype_ok(dy_dtype) || !(kept || dtype_ok(x_dtype)) || !dtype_ok(a_dtype) || !dtype_ok(dx_dtype))
        return CONVIMG_ERR_DTYPE;
    if (lddy < N || (!kept && ldx < K))
        return CONVIMG_ERR_SHAPE;
    if (!ddown || !dup || !ws || (wt_codes && !wt_scales)
        || (M > 0 && (!dy || !x || (kept && !x_scales) || !down || !up || !scale || !ids || !h || (!dx) != (!wt_codes))))
        return CONVIMG_ERR_NULL;
    if (misaligned(ws, 16) || misaligned(wt_codes, 16) || misaligned(wt_scales, 4)
        || (kept && (misaligned(x, 16) || misaligned(x_scales, 4))))
        return CONVIMG_ERR_ALIGN;
    const AdBwdLayout l = ad_bwd_layout(M, N, K, adapters, rank);
    if (ws_bytes < l.total)
        return CONVIMG_ERR_WORKSPACE;
    const size_t na = (size_t)adapters * rank, ab = dtype_bytes(a_dtype);
    const void *in[10] = {dy, x, kept ? x_scales : nullptr, wt_codes, wt_scales, down, up, scale, ids, h},
               *outs[4] = {dx, ddown, dup, ws};
    const size_t nin[10] = {span_bytes(M, lddy, N, dy_dtype), kept ? mxi_code_bytes(M, K) : span_bytes(M, ldx, K, x_dtype),
                            mxi_scale_bytes(M, K), mx_code_bytes(K, N), mx_scale_bytes(K, N), na * K * ab, na * N * ab,
                            (size_t)adapters * 4, (size_t)M * 4, (size_t)M * rank * 4},
                 nout[4] = {span_bytes(M, K, K, dx_dtype), na * K * 4, na * N * 4, l.total};
    if (any_overlap(outs, nout, 4, in, nin, 10))
        return CONVIMG_ERR_ALIAS;
    if (M == 0) {
        fill_zero(ddown, (long long)(na * K), stream);
        fill_zero(dup, (long long)(na * N), stream);
        return launched();
    }
    unsigned char *base = (unsigned char *)ws, *codes = base + l.dy, *scales = codes + align256(mx_code_bytes(M, N));
    float *t = (float *)(base + l.t);
    int *order = (int *)(base + l.order), *key = order + 2LL * M, *start = (int *)(base + l.start),
        *nan = (int *)(base + l.nan);
    adapter_sort(ids, M, adapters, order, key, start, nan, stream);
    unsigned char *terms = dx ? base + l.terms : nullptr;
    const AdShrinkArgs s = {dy, up, scale, key, order, start, t, terms, nullptr, dx ? codes : nullptr, scales, nullptr, nullptr,
                            lddy, M, N, adapters, rank};
    adapter_shrink(s, {false, true}, dy_dtype, a_dtype, stream);
    if (dx) {
        const MxAdapterArgs ad = {terms, t, down, scale, key, order, adapters, rank, a_dtype};
        gemm_adapters(gemm_args({codes, scales}, {(const unsigned char *)wt_codes, (const unsigned char *)wt_scales},
                                nullptr, M, K, N, dx),
                      ad, dx_dtype, stream);
    }
    const int rt = grad_chunks_of_ranks(rank);
    const AdGradArgs up_args = {h,   dy,   nullptr, order, key, start, scale, dup, (float *)(base + l.part_up), nan, lddy, M, N,
                                adapters, rank, 0, rank, l.per_up, ad_chunks(M, l.per_up), grad_tiles(N), rt},
                     down_args = {t, x, (const unsigned char *)x_scales, order, key, start, scale, ddown,
                                  (float *)(base + l.part_down), nan, ldx, M, K, adapters, rank, 1, adapter_ranks(rank),
                                  l.per_down, ad_chunks(M, l.per_down), grad_tiles(K), rt};
    auto grads = dy_dtype == CONVIMG_BF16 ? adapter_grads_bf16 : dy_dtype == CONVIMG_FP16 ? adapter_grads_fp16 : adapter_grads_fp32;
    grads(up_args, down_args, x_dtype, stream);
    return launched();
}

}  // extern "C"
