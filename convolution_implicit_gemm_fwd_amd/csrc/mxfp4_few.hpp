// mxfp4_few.hpp -- the product of a few dense rows (decoding) with MXFP4
// weights in one launch.
//
// Reading the weights once is all the work, so a workgroup takes 16 columns
// of the output, its waves share the contracted axis, and each wave keeps
// three stages of 256 k in flight to LDS: whole cache lines, eight lanes a row
// (loading the matrix instruction's operands straight into registers puts
// neighbouring lanes on different rows and reaches half the rate).  Every
// workgroup quantises the rows into LDS for itself while its first weights
// arrive.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes one block (32 consecutive k) of row
// lane % 16 from each lane, block lane / 16 of the step's four; a lane ends
// with four neighbouring columns of one output row, and the waves' sums meet
// in LDS in a fixed order.
//
// One row through 4096 x 4096: 3.9 to 4.4 us a call, back to back, of which an
// empty launch takes 1.9 and the 8.9 MB 1.7 at a copy's rate; 8192 x 8192 9.8 us.
// In two launches (quantise, product) 7.4 and 13.9 us.
#pragma once

#include "mxfp4_gemm.hpp"

namespace convimg {

constexpr int kMxFewWaves = 8, kMxFewRing = 3;
constexpr int kMxFewM = 4, kMxFewSize = 1 << 15;      // rows and elements at most

// LDS: a row of codes ends in 16 bytes that set the rows' banks apart.
constexpr int kMxFewRows = kMxFewSize / 2 + kMxFewM * (64 + 16) + (kMxFewSize / 128 + kMxFewM) * 4;
constexpr int kMxFewStage = 16 * 128 + 256;

struct MxFewArgs {
    const void *x;                  // dense rows ldx apart
    const unsigned char *w, *sw;    // codes [N][kb * 16], scales [quads][N][4]
    const float *bias;
    void *out;                      // [M][N]
    long long ldx;
    int M, N, K, kb;
};

template <typename X, typename O>
__global__ __launch_bounds__(kMxFewWaves * 64) void mx_gemm_few(MxFewArgs g)
{
    __shared__ __attribute__((aligned(16))) unsigned char rows[kMxFewRows];
    __shared__ __attribute__((aligned(16))) unsigned char ring[kMxFewWaves][kMxFewRing][kMxFewStage];
    constexpr int PER = 3;                      // copies a stage
    const int lane = threadIdx.x & 63, r16 = lane & 15, b4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int n0 = blockIdx.x * 16;
    const int quads = (g.kb + 3) / 4, pairs = (quads + 1) / 2;

    const __amdgpu_buffer_rsrc_t rw =
        __builtin_amdgcn_make_buffer_rsrc((void *)g.w, 0, (unsigned)g.N * g.kb * 16u, kMxRsrcWord3);
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc((void *)g.sw, 0, (unsigned)g.N * quads * 4u, kMxRsrcWord3);

    // Stage of the pair p of scale dwords (256 k): 16 rows of eight chunks,
    // chunk c of row r at c ^ (r / 2 % 8), then the scale dwords [2][16].
    // Zeros past the operand, later pairs included.
    auto fetch = [&](int p, int u) {
        unsigned char *s = ring[wave][u];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = i * 8 + (lane >> 3), blk = p * 8 + ((lane & 7) ^ ((r >> 1) & 7)), n = n0 + r;
            mx_dma16(rw, s + i * 1024,
                     n < g.N && blk < g.kb ? ((unsigned)n * (unsigned)g.kb + blk) * 16u : kMxOutOfRange);
        }
        const int q = p * 2 + (b4 & 1), n = n0 + r16;
        mx_dma4(rs, s + 2048, lane < 32 && n < g.N && q < quads ? ((unsigned)q * g.N + n) * 4u : kMxOutOfRange);
    };

    const int pitch = quads * 64 + 16, last = quads * 128, nt = blockDim.x * 8;
    unsigned char *scales = rows + g.M * pitch;
    // (the rows are fetched before the weights, as loads return in order; what
    // does not fit these registers is late)
    constexpr int AHEAD = 4;
    const int per = (last + nt - 1) / nt;      // a row's passes of all threads
    Raw8<X> raw[AHEAD];
    auto load_row = [&](int i, Raw8<X> &r) {
        const int m = i / per, c = (i - m * per) * nt + threadIdx.x * 8;
        r = load_raw8<X>((const typename X::raw *)g.x + m * g.ldx, c, g.K);
    };
    auto quantise = [&](int i, const Raw8<X> &r) {
        const int m = i / per, c = (i - m * per) * nt + threadIdx.x * 8;
        float v[8];
        unpack8<X>(tail8<X>(r, c, g.K), v);
        unsigned top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top = mx_top(top, v[e]);
        const unsigned byte = mx_scale_byte(quad_max(top));
        if (c < last) {
            *(unsigned *)(rows + m * pitch + c / 2) = mx_encode8(v, mx_scale_value(byte));
            if ((c & 31) == 0)
                scales[((c >> 7) * g.M + m) * 4 + ((c >> 5) & 3)] = (unsigned char)byte;
        }
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (i < g.M * per)
            load_row(i, raw[i]);
#pragma unroll
    for (int u = 0; u < kMxFewRing; ++u)
        fetch(u * waves + wave, u);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (i < g.M * per)
            quantise(i, raw[i]);
    for (int i = AHEAD; i < g.M * per; ++i) {
        load_row(i, raw[0]);
        quantise(i, raw[0]);
    }
    mx_wait_lds();
    mx_barrier();

    f32x4_t acc = {};
    for (int p0 = wave; p0 < pairs; p0 += kMxFewRing * waves) {
#pragma unroll
        for (int u = 0; u < kMxFewRing; ++u) {
            const int p = p0 + u * waves;
            mx_wait_vm<(kMxFewRing - 1) * PER>();
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
            const unsigned char *s = ring[wave][u];
            i32x4_t w[2], x[2];
            unsigned sw[2], sx[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // (rows past M give rows of the product that nobody stores,
                // steps past K meet zero weights)
                const int m = min(r16, g.M - 1), q = min(2 * p + h, quads - 1);
                w[h] = *(const i32x4_t *)(s + r16 * 128 + (((h * 4 + b4) ^ ((r16 >> 1) & 7)) * 16));
                sw[h] = *(const unsigned *)(s + 2048 + (h * 16 + r16) * 4);
                x[h] = *(const i32x4_t *)(rows + m * pitch + q * 64 + b4 * 16);
                sx[h] = *(const unsigned *)(scales + (q * g.M + m) * 4);
            }
            mx_wait_lds();
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
            fetch(p + kMxFewRing * waves, u);      // the stage has been read
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const i32x8_t a8 = {w[h][0], w[h][1], w[h][2], w[h][3], 0, 0, 0, 0};
                const i32x8_t b8 = {x[h][0], x[h][1], x[h][2], x[h][3], 0, 0, 0, 0};
                acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, acc, 4, 4, 0, (int)(sw[h] >> (8 * b4)),
                                                                       0, (int)(sx[h] >> (8 * b4)));
            }
        }
    }
    mx_wait_vm<0>();

    // the waves' sums, in order; a wave's lie in its own ring
    if (r16 < g.M)
        *(f32x4_t *)(ring[wave][0] + (r16 * 16 + b4 * 4) * 4) = acc;
    mx_wait_lds();
    mx_barrier();
    for (int e = threadIdx.x; e < g.M * 16; e += blockDim.x) {
        const int n = n0 + (e & 15);
        if (n < g.N) {
            float s = g.bias ? g.bias[n] : 0.f;
            for (int k = 0; k < waves; ++k)
                s += *(const float *)(ring[k][0] + e * 4);
            store1<O>((typename O::raw *)g.out + (long long)(e >> 4) * g.N + n, s);
        }
    }
}

}  // namespace convimg
