// mxfp4_plan.hpp -- host side shared by the products of MXFP4 rows: packed
// operands in a workspace and the choice of a product's shape.
#pragma once

#include "mxfp4_few.hpp"

namespace convimg {

struct MxOperand {
    const unsigned char *codes, *scales;
};

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Bytes of one packed operand in a workspace.
inline size_t packed_bytes(int rows, int cols)
{
    return align256(mx_code_bytes(rows, cols)) + align256(mx_scale_bytes(rows, cols));
}

inline unsigned eights(long long n) { return (unsigned)((n + 7) / 8 * 8); }

inline unsigned row_grid(int rows, int lg) { return (unsigned)(((long long)rows + (kMxThreads >> lg) - 1) / (kMxThreads >> lg)); }

inline long long tile_count(int M, int N, int bm, int bn) { return (long long)((M + bm - 1) / bm) * ((N + bn - 1) / bn); }

inline auto tiles_of(int M, int N)
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
// With adapters beside the product, which cost the smaller tiles waves, the same
// bounds hold (16 ranks, the whole call): 64x4096x4096 12.1 in 32 x 32 against 13.2
// in 64 x 32; 256 rows 18.6 in 64 x 64 against 21.9 in 128 x 64 and 23.2 in 64 x 32;
// 512 rows 28.9 in 128 x 64 against 30.0 and 32.7; 1024 rows 34.9 in 128 x 128
// against 41.0 and 47.4; 4096 rows 65.2 in 256 x 256 against 72.7; short ones within
// 4 %: 8192x8192x256 73.2 against 72.1 in 256 x 256, x512 82.0 against 80.0 in the
// longer 128 x 128.
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
inline int shape_level(Shape s) { return s <= k128 ? s : s - 1; }

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

inline MxGemmArgs gemm_args(MxOperand a, MxOperand b, const float *bias, int M, int N, int K, void *out)
{
    return {a.codes, b.codes, a.scales, b.scales, bias, out, M, N, mx_blocks(K), 0, 0};
}

inline unsigned gemm_grid(MxGemmArgs &g, int bm, int bn)
{
    g.tm = (g.M + bm - 1) / bm;
    g.tn = (g.N + bn - 1) / bn;
    return eights((long long)g.tm * g.tn);
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
inline bool few_dense(int M, int K) { return M <= kMxFewM && (long long)M * K <= kMxFewSize; }

inline int launched() { return hipGetLastError() == hipSuccess ? CONVIMG_OK : CONVIMG_ERR_LAUNCH; }

inline bool misaligned(const void *p, unsigned n) { return ((uintptr_t)p & (n - 1)) != 0; }

// Quantises rows into packed ones (mxfp4.hip).
void quantize(const void *x, long long ldx, int rows, int cols, int dtype, unsigned char *codes,
              unsigned char *scales, hipStream_t stream);
// Fills n floats with zeros (mxfp4.hip).
void fill_zero(float *p, long long n, hipStream_t stream);

}  // namespace convimg
