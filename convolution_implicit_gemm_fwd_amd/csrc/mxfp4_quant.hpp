// mxfp4_quant.hpp -- dense rows to MXFP4 and back.
//
// Blocks along a row are quantised straight from memory (four neighbouring
// lanes hold one).  Blocks down the columns go through LDS in tiles of 128 x
// 128 (four blocks either way, so that a tile owns whole scale dwords); a
// tile can also be quantised along its rows and summed down its columns, so
// that an operand that is contracted over either axis is read once.
//
// Both are bound by memory: 8192 x 8192 bf16 along the rows 36 us, down the
// columns 36 us (170 MB, 4.7 TB/s; a copy of 256 MiB reaches 5.2).
#pragma once

#include "mxint8.hpp"

namespace convimg {

constexpr int kMxThreads = 256;

struct MxQuantArgs {
    const void *x;
    unsigned char *codes, *scales;
    long long ldx;
    int rows, cols;        // of x
    int lg;                // log2 of the threads a row
};

// Place of a workgroup in a launch whose grid is a multiple of 8: each of the
// 8 XCDs, which take workgroups in turn, gets one run of places, so that the
// parts of a cache line that neighbours write or read meet in one L2.
__device__ __forceinline__ unsigned mx_xcd_tile(unsigned block, unsigned blocks)
{
    return (block & 7) * (blocks >> 3) + (block >> 3);
}

// Rows to MXFP4: a thread takes 8 columns, of up to four groups at once;
// 1 << lg threads a row, at least 16 where a row has more than 64 columns, so
// that a scale dword is written whole.
template <typename T>
__global__ __launch_bounds__(kMxThreads) void mx_quantize_rows(MxQuantArgs a)
{
    constexpr int U = 4;
    const int tpr = 1 << a.lg;
    const long long row =
        (long long)mx_xcd_tile(blockIdx.x, gridDim.x) * (kMxThreads >> a.lg) + (threadIdx.x >> a.lg);
    if (row >= a.rows)
        return;
    const typename T::raw *x = (const typename T::raw *)a.x + row * a.ldx;
    const int kp = (a.cols + 31) & ~31, end = a.lg >= 4 ? (a.cols + 127) & ~127 : tpr * 8;
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
            unsigned top = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                top = mx_top(top, v[e]);
            top = quad_max(top);
            const unsigned byte = mx_scale_byte(top);
            if (c < kp)
                ((unsigned *)a.codes)[row * (kp / 8) + c / 8] = mx_encode8(v, mx_scale_value(byte));
            const unsigned word = a.lg >= 4   ? mx_scale_word<16>(byte, c >> 5)
                                  : a.lg == 3 ? mx_scale_word<8>(byte, c >> 5)
                                              : mx_scale_word<4>(byte, c >> 5);
            if ((c & 127) == 0)
                ((unsigned *)a.scales)[(long long)(c >> 7) * a.rows + row] = word;
        }
    }
}

// A matrix that is quantised in tiles: down its columns into ccodes
// [cols][rows / 32 blocks], along its rows into rcodes, and summed down its
// columns, one partial sum a row of tiles.
// An operand kept in 8 bits is given by its codes and xs, its scale bytes.
struct MxTileArgs {
    const void *x;
    const unsigned char *xs;
    long long ldx;
    int rows, cols;
    unsigned char *ccodes, *cscales, *rcodes, *rscales;
    float *part;           // [tiles down][cols]
};

constexpr int kMxTile = 128, kMxTileThreads = 512;
constexpr int kMxOutPitch = 64 + 16;      // LDS bytes of a column's result: four blocks of codes, their scales

template <typename T>
constexpr int mx_tile_pitch() { return kMxTile * (int)sizeof(typename T::raw) + 16; }

template <typename T>
constexpr int mx_tile_lds() { return kMxTile * mx_tile_pitch<T>(); }      // (the results, 96 bytes a column, take its place)

inline long long mx_tiles(int rows, int cols)
{
    return (long long)((rows + kMxTile - 1) / kMxTile) * ((cols + kMxTile - 1) / kMxTile);
}

// 32 values to four code dwords and a scale byte.
__device__ __forceinline__ unsigned mx_encode32(const float (&v)[32], u32v4_t &q)
{
    unsigned top = 0;
#pragma unroll
    for (int e = 0; e < 32; ++e)
        top = mx_top(top, v[e]);
    const unsigned byte = mx_scale_byte(top);
    const float scale = mx_scale_value(byte);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float w[8] = {v[8 * i],     v[8 * i + 1], v[8 * i + 2], v[8 * i + 3],
                            v[8 * i + 4], v[8 * i + 5], v[8 * i + 6], v[8 * i + 7]};
        q[i] = mx_encode8(w, scale);
    }
    return byte;
}

// Eight values of a row kept in 8 bits as bf16, which holds them exactly.
__device__ __forceinline__ Raw8<Bf16> load_kept8(const MxTileArgs &a, int row, int col)
{
    Raw8<Bf16> r = {};
    if (row < a.rows && col < a.cols) {
        const int kp = (a.cols + 31) & ~31;
        float v[8];
        mxi_decode8(*(const uint2 *)((const unsigned char *)a.x + (long long)row * kp + col),
                    mxi_unit(a.xs, row, a.cols, col), v);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            r.w[0][e] = pack_bf16(v[2 * e], v[2 * e + 1]);
    }
    return r;
}

// One tile, by the whole workgroup; lds: mx_tile_lds<T>() bytes, 16-byte
// aligned.  ROWS: along the rows and the column sums too.  KEPT: of an operand
// in 8 bits, which is bf16 from there on.
template <typename T, bool ROWS, bool KEPT = false>
__device__ __forceinline__ void mx_quantize_tile(const MxTileArgs &a, unsigned tile, unsigned char *lds)
{
    constexpr int PITCH = mx_tile_pitch<T>(), ES = sizeof(typename T::raw);
    static_assert(kMxTile * (kMxOutPitch + 16) <= mx_tile_lds<T>(), "results fit the tile");
    float *sums = (float *)(lds + kMxTile * kMxOutPitch);      // [4 waves][128]
    const int across = (a.cols + kMxTile - 1) / kMxTile;
    // Two rows of tiles side by side: the halves of a cache line of codes, down
    // and along, are written by tiles that run at about the same time.
    const int tiles_down = (a.rows + kMxTile - 1) / kMxTile;
    const int pr = (int)(tile / (2u * across)), in = (int)(tile - (unsigned)pr * 2u * across);
    const bool two = pr * 2 + 1 < tiles_down;
    const int tr = pr * 2 + (two ? in & 1 : 0), tc = two ? in >> 1 : in;
    const int r0 = tr * kMxTile, c0 = tc * kMxTile;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;

    // 16 threads a row of the tile, zeros past the matrix.  Whole tiles, which
    // need no test a load, have all loads in flight at once.
    constexpr int PASSES = kMxTile * 16 / kMxTileThreads, LR = kMxTileThreads / 16;
    const bool whole = r0 + kMxTile <= a.rows && c0 + kMxTile <= a.cols;
    const int lr = t >> 4, lc = (t & 15) * 8;
    Raw8<T> raw[PASSES];
    if constexpr (KEPT) {
        static_assert(!ROWS && T::code == CONVIMG_BF16, "bf16 values, down the columns");
#pragma unroll
        for (int p = 0; p < PASSES; ++p)
            raw[p] = load_kept8(a, r0 + lr + p * LR, c0 + lc);
    } else if (whole) {
        const typename T::raw *x = (const typename T::raw *)a.x + (long long)(r0 + lr) * a.ldx + c0 + lc;
#pragma unroll
        for (int p = 0; p < PASSES; ++p)
            raw[p] = load_raw8<T>(x + (long long)p * LR * a.ldx, 0, 8);
    } else {
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            raw[p] = {};
            if (r0 + lr + p * LR < a.rows)
                raw[p] = load_raw8<T>((const typename T::raw *)a.x + (long long)(r0 + lr + p * LR) * a.ldx, c0 + lc,
                                      a.cols);
        }
#pragma unroll
        for (int p = 0; p < PASSES; ++p)
            raw[p] = tail8<T>(raw[p], c0 + lc, a.cols);
    }
#pragma unroll
    for (int p = 0; p < PASSES; ++p)
        *(Raw8<T> *)(lds + (p * LR + lr) * PITCH + lc * ES) = raw[p];
    __syncthreads();

    // down: a wave takes 32 rows of 64 columns, a lane one column
    const int blk = wave & 3, c = (wave >> 2) * 64 + lane;
    u32v4_t down;
    unsigned byte;
    float sum = 0.f;
    {
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            v[e] = load1<T>((const typename T::raw *)(lds + (blk * 32 + e) * PITCH + c * ES));
            sum += v[e];
        }
        byte = mx_encode32(v, down);
    }
    // along: a thread takes a block of a row
    if constexpr (ROWS) {
        const int row = r0 + (t >> 2), nb = mx_blocks(a.cols), b0 = tc * 4 + (t & 3);
        float v[32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Raw8<T> w = *(const Raw8<T> *)(lds + (t >> 2) * PITCH + ((t & 3) * 32 + i * 8) * ES);
            float u[8];
            unpack8<T>(w, u);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[i * 8 + e] = u[e];
        }
        u32v4_t q;
        unsigned word = mx_encode32(v, q) << (8 * (t & 3));
        if (row < a.rows && b0 < nb)
            *(u32v4_t *)(a.rcodes + ((long long)row * nb + b0) * 16) = q;
        word |= (unsigned)__builtin_amdgcn_mov_dpp((int)word, 0xB1, 0xf, 0xf, true);
        word |= (unsigned)__builtin_amdgcn_mov_dpp((int)word, 0x4E, 0xf, 0xf, true);
        if (row < a.rows && (t & 3) == 0)
            *(unsigned *)(a.rscales + ((long long)tc * a.rows + row) * 4) = word;
    }
    __syncthreads();      // the tile has been read
    *(u32v4_t *)(lds + c * kMxOutPitch + blk * 16) = down;
    lds[c * kMxOutPitch + 64 + blk] = (unsigned char)byte;
    if constexpr (ROWS)
        sums[blk * kMxTile + c] = sum;
    __syncthreads();

    // the columns' results, four lanes a column
    {
        const int col = c0 + (t >> 2), nb = mx_blocks(a.rows), b0 = tr * 4 + (t & 3);
        const unsigned char *o = lds + (t >> 2) * kMxOutPitch;
        if (col < a.cols) {
            if (b0 < nb)
                *(u32v4_t *)(a.ccodes + ((long long)col * nb + b0) * 16) = *(const u32v4_t *)(o + (t & 3) * 16);
            if ((t & 3) == 0)
                *(unsigned *)(a.cscales + ((long long)tr * a.cols + col) * 4) = *(const unsigned *)(o + 64);
        }
        if constexpr (ROWS)
            if (t < kMxTile && c0 + t < a.cols)
                a.part[(long long)tr * a.cols + c0 + t] =
                    (sums[t] + sums[kMxTile + t]) + (sums[2 * kMxTile + t] + sums[3 * kMxTile + t]);
    }
}

// The tiles first .. end - 1.
template <typename T>
__global__ __launch_bounds__(kMxTileThreads) void mx_quantize_cols(MxTileArgs a, unsigned first, unsigned end)
{
    __shared__ __attribute__((aligned(16))) unsigned char lds[mx_tile_lds<T>()];
    const unsigned tile = first + mx_xcd_tile(blockIdx.x, gridDim.x);
    if (tile < end)
        mx_quantize_tile<T, false>(a, tile, lds);
}

// The operands of the backward pass in one launch: dy both ways with its
// column sums, w and x down their columns (8192x4096x4096 bf16: 46 us for 232
// MB, 5.0 TB/s).
// KEPT: x is kept in 8 bits; X is then w's type alone.
template <typename DY, typename X, bool KEPT>
__global__ __launch_bounds__(kMxTileThreads) void mx_quantize_bwd(MxTileArgs dy, MxTileArgs w, MxTileArgs x,
                                                              unsigned dy_tiles, unsigned w_tiles, unsigned x_tiles)
{
    constexpr int LDS = mx_tile_lds<DY>() > mx_tile_lds<X>() ? mx_tile_lds<DY>() : mx_tile_lds<X>();
    __shared__ __attribute__((aligned(16))) unsigned char lds[LDS];
    // (each operand's tiles spread over all XCDs; the blocks of each are a
    // multiple of 8)
    const unsigned dy_blocks = (dy_tiles + 7) & ~7u, w_blocks = (w_tiles + 7) & ~7u;
    if (blockIdx.x < dy_blocks) {
        const unsigned tile = mx_xcd_tile(blockIdx.x, dy_blocks);
        if (tile < dy_tiles)
            mx_quantize_tile<DY, true>(dy, tile, lds);
        return;
    }
    const unsigned b = blockIdx.x - dy_blocks;
    const bool is_w = b < w_blocks;
    const unsigned tile = is_w ? mx_xcd_tile(b, w_blocks) : mx_xcd_tile(b - w_blocks, (x_tiles + 7) & ~7u);
    if constexpr (KEPT) {
        if (is_w && tile < w_tiles)
            mx_quantize_tile<X, false>(w, tile, lds);
        else if (!is_w && tile < x_tiles)
            mx_quantize_tile<Bf16, false, true>(x, tile, lds);
    } else if (tile < (is_w ? w_tiles : x_tiles)) {
        mx_quantize_tile<X, false>(is_w ? w : x, tile, lds);
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

}  // namespace convimg
