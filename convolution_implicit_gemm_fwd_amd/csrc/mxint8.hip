// mxint8.hip -- activations to 8-bit rows and back (mxint8.hpp).
//
// Both are bound by memory: a bf16 value costs 2 bytes and 33 / 32.  16384 x
// 4101 in bf16, rows 11 values apart: 41.4 us to 8 bits (206 MB, 5.0 TB/s), 33.3
// us back (208 MB, 6.3 TB/s; a copy runs at 5.4); 1 x 4096 1.8 us, a launch.
#include "mxint8.hpp"

namespace convimg {

constexpr int kMxiThreads = 256;

struct MxiArgs {
    const void *x;
    unsigned char *codes, *scales;
    void *out;
    long long rows, ldx;
    int cols;
    int lg;                // log2 of the threads a row
};

// A thread takes 8 columns of up to four groups at once; at least 16 threads a
// row where a row has more than 64 columns, so that a scale dword is written whole.
template <typename T>
__global__ __launch_bounds__(kMxiThreads) void mxi_quantize_rows(MxiArgs a)
{
    constexpr int U = 4;
    const int tpr = 1 << a.lg, end = a.lg >= 4 ? (a.cols + 127) & ~127 : tpr * 8;
    const long long step = (long long)gridDim.x * (kMxiThreads >> a.lg);
    for (long long row = (long long)blockIdx.x * (kMxiThreads >> a.lg) + (threadIdx.x >> a.lg); row < a.rows; row += step) {
        const typename T::raw *x = (const typename T::raw *)a.x + row * a.ldx;
        for (int c0 = (threadIdx.x & (tpr - 1)) * 8; c0 < end; c0 += U * tpr * 8) {
            Raw8<T> raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c0 + u * tpr * 8 < end)
                    raw[u] = load_raw8<T>(x, c0 + u * tpr * 8, a.cols);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * tpr * 8;
                if (c >= end)      // (lanes of 128 columns agree on this)
                    break;
                float v[8];
                unpack8<T>(tail8<T>(raw[u], c, a.cols), v);
                if (a.lg >= 4)
                    mxi_emit8<16>(a.codes, (unsigned *)a.scales, row, a.cols, c, v);
                else if (a.lg == 3)
                    mxi_emit8<8>(a.codes, (unsigned *)a.scales, row, a.cols, c, v);
                else
                    mxi_emit8<4>(a.codes, (unsigned *)a.scales, row, a.cols, c, v);
            }
        }
    }
}

template <typename T>
__global__ __launch_bounds__(kMxiThreads) void mxi_dequantize_rows(MxiArgs a)
{
    constexpr int U = 4;
    const int tpr = 1 << a.lg, kp = (a.cols + 31) & ~31;
    const long long step = (long long)gridDim.x * (kMxiThreads >> a.lg);
    for (long long row = (long long)blockIdx.x * (kMxiThreads >> a.lg) + (threadIdx.x >> a.lg); row < a.rows; row += step) {
        for (int c0 = (threadIdx.x & (tpr - 1)) * 8; c0 < a.cols; c0 += U * tpr * 8) {
            uint2 q[U];
            float unit[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * tpr * 8;
                if (c < a.cols) {
                    q[u] = *(const uint2 *)(a.codes + row * kp + c);
                    unit[u] = mxi_unit(a.scales, row, a.cols, c);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * tpr * 8;
                if (c >= a.cols)
                    break;
                float v[8];
                mxi_decode8(q[u], unit[u], v);
                store8<T>((typename T::raw *)a.out + row * a.cols, c, a.cols, v);
            }
        }
    }
}

// A launch holds fewer than 2^32 threads; more rows are walked in strides.
unsigned mxi_grid(long long rows, int lg)
{
    const long long n = (rows + (kMxiThreads >> lg) - 1) / (kMxiThreads >> lg);
    return (unsigned)(n < (1 << 22) ? n : (1 << 22));
}

int mxi_shape(long long rows, int cols)
{
    if (rows < 0 || cols <= 0)
        return CONVIMG_ERR_SHAPE;
    return rows > kMaxRows || cols > kMaxCols ? CONVIMG_ERR_RANGE : CONVIMG_OK;
}

bool mxi_misaligned(const void *codes, const void *scales) { return ((uintptr_t)codes & 15) || ((uintptr_t)scales & 3); }

int mxi_launched() { return hipGetLastError() == hipSuccess ? CONVIMG_OK : CONVIMG_ERR_LAUNCH; }

}  // namespace convimg

using namespace convimg;

extern "C" {

int mxint8_bytes(long long rows, int cols, size_t *codes, size_t *scales)
{
    if (!codes || !scales)
        return CONVIMG_ERR_NULL;
    const int rc = mxi_shape(rows, cols);
    if (rc != CONVIMG_OK)
        return rc;
    *codes = mxi_code_bytes(rows, cols);
    *scales = mxi_scale_bytes(rows, cols);
    return CONVIMG_OK;
}

int mxint8_quantize(const void *x, long long ldx, long long rows, int cols, int dtype, void *codes, void *scales,
                    hipStream_t stream)
{
    if (rows < 0 || cols <= 0 || ldx < cols)
        return CONVIMG_ERR_SHAPE;
    if (!dtype_ok(dtype))
        return CONVIMG_ERR_DTYPE;
    const int rc = mxi_shape(rows, cols);
    if (rc != CONVIMG_OK || rows == 0)
        return rc;
    if (!x || !codes || !scales)
        return CONVIMG_ERR_NULL;
    if (mxi_misaligned(codes, scales))
        return CONVIMG_ERR_ALIGN;
    const size_t nx = span_bytes(rows, ldx, cols, dtype), nc = mxi_code_bytes(rows, cols), ns = mxi_scale_bytes(rows, cols);
    if (row_overlaps(codes, nc, x, nx) || row_overlaps(scales, ns, x, nx) || row_overlaps(codes, nc, scales, ns))
        return CONVIMG_ERR_ALIAS;
    const int lg = row_lg(cols);
    const MxiArgs a = {x, (unsigned char *)codes, (unsigned char *)scales, nullptr, rows, ldx, cols, lg};
    with_dtype(dtype, [&](auto t) {
        hipLaunchKernelGGL(mxi_quantize_rows<decltype(t)>, dim3(mxi_grid(rows, lg)), dim3(kMxiThreads), 0, stream, a);
    });
    return mxi_launched();
}

int mxint8_dequantize(const void *codes, const void *scales, long long rows, int cols, int dtype, void *out,
                      hipStream_t stream)
{
    const int rc = mxi_shape(rows, cols);
    if (rc != CONVIMG_OK)
        return rc;
    if (!dtype_ok(dtype))
        return CONVIMG_ERR_DTYPE;
    if (rows == 0)
        return CONVIMG_OK;
    if (!codes || !scales || !out)
        return CONVIMG_ERR_NULL;
    if (mxi_misaligned(codes, scales))
        return CONVIMG_ERR_ALIGN;
    const size_t no = span_bytes(rows, cols, cols, dtype);
    if (row_overlaps(out, no, codes, mxi_code_bytes(rows, cols))
        || row_overlaps(out, no, scales, mxi_scale_bytes(rows, cols)))
        return CONVIMG_ERR_ALIAS;
    const int lg = row_lg(cols);
    const MxiArgs a = {nullptr, (unsigned char *)codes, (unsigned char *)scales, out, rows, 0, cols, lg};
    with_dtype(dtype, [&](auto t) {
        hipLaunchKernelGGL(mxi_dequantize_rows<decltype(t)>, dim3(mxi_grid(rows, lg)), dim3(kMxiThreads), 0, stream, a);
    });
    return mxi_launched();
}

}  // extern "C"
