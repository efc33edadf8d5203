// mxfp4_gemm.hpp -- products of MXFP4 rows: out = a b^T + bias for a [M][K],
// b [N][K] in 32-value blocks along K (the layout of mxfp4_quantize).
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes from each lane 32 consecutive k of
// one row, which is one block, with its scale byte picked out of a dword, so
// a dword of four scale bytes serves 128 k.  b's rows are the instruction's
// rows, so that a lane ends with four neighbouring columns of one output row.
//
// 8192^3 takes 260 us (4.2 PFLOP/s) on normal data and 222 us on zeros.  The
// same stream of matrix instructions alone, operands held in registers, takes
// 201 us (5.5 PFLOP/s) and 156 us: the clock falls with the power that the
// data's toggling draws.  With the operands' reads from LDS it takes 195 and
// 164 us (the same K tiles over and over), so the copies into LDS are what
// costs 60 us more, on either data.  A K tile of 256 copies 68 KB a workgroup
// and reads 131 KB, and the largest wave tile that the registers hold (128 x
// 128) bounds what is left.  Fetching the lines into L2 two K tiles ahead of
// the copies changes nothing.
#pragma once

#include "mxfp4_quant.hpp"

namespace convimg {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr unsigned kMxOutOfRange = 0x80000000u;   // buffer offset past every packed operand
constexpr int kMxRsrcWord3 = 0x00020000;          // raw buffer, 32-bit data format

struct MxGemmArgs {
    const unsigned char *a, *b;     // codes: a [M][kb * 16], b [N][kb * 16]
    const unsigned char *sa, *sb;   // scales: [quads][M or N][4]
    const float *bias;              // [N] or NULL
    void *out;                      // [M][N]
    int M, N, kb;                   // kb: blocks of 32 along the contracted axis
    int tm, tn;                     // tiles along M and N
};

// s_waitcnt vmcnt(N) alone (gfx9 encoding; 7 and 15 leave the other counters
// unconstrained).
template <int N>
__device__ __forceinline__ void mx_wait_vm()
{
    static_assert(N >= 0 && N < 64, "vmcnt is 6 bits");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

__device__ __forceinline__ void mx_wait_lds() { __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4)); }

__device__ __forceinline__ void mx_barrier()
{
    __atomic_signal_fence(__ATOMIC_SEQ_CST);   // no compiler motion of LDS accesses across
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

__device__ __forceinline__ void mx_dma16(__amdgpu_buffer_rsrc_t r, unsigned char *lds, unsigned off)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)lds, 16, off, 0, 0, 0);
}

__device__ __forceinline__ void mx_dma4(__amdgpu_buffer_rsrc_t r, unsigned char *lds, unsigned off)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)lds, 4, off, 0, 0, 0);
}

// Byte `sel` (known when compiled) of each scale dword.
__device__ __forceinline__ f32x16_t mx_mfma32(int sel, i32x4_t b, i32x4_t a, f32x16_t c, int sb, int sa)
{
    const i32x8_t b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0}, a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
    switch (sel) {
    case 0: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b8, a8, c, 4, 4, 0, sb, 0, sa);
    case 1: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b8, a8, c, 4, 4, 1, sb, 1, sa);
    case 2: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b8, a8, c, 4, 4, 2, sb, 2, sa);
    default: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b8, a8, c, 4, 4, 3, sb, 3, sa);
    }
}

// Tile number `id` (mx_xcd_tile: each XCD takes one run of them, so that its
// L2 serves neighbours), in groups of 8 tile rows so that the tiles in flight
// are near square.
__device__ __forceinline__ void mx_tile(const MxGemmArgs &g, int id, int &m, int &n)
{
    const int span = 8 * g.tn, group = id / span, in = id - group * span;
    const int rows = min(g.tm - group * 8, 8);
    n = in / rows;
    m = group * 8 + in - n * rows;
}

// A kernel's shape: tile, waves along M and N, K tile, stages, groups of waves
// along K.
template <int BM_, int BN_, int WM_, int WN_, int BK_, int STAGES_, int KG_>
struct GemmShape {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = BK_, STAGES = STAGES_, KG = KG_;
    // LDS: rows of codes, and scale dwords in slots of 64 rows
    static constexpr int SLOTS = (BM + 63) / 64 + (BN + 63) / 64;
    static constexpr int CODES = (BM + BN) * (BK / 2), STAGE = CODES + SLOTS * 256 * (BK / 128);
    static constexpr int threads = WM * WN * KG * 64;
};

template <typename S, int OS>
constexpr int mx_gemm_lds()
{
    constexpr int ring = S::KG * S::STAGES * S::STAGE, rows = S::WM * S::WN * 32 * (S::BN / S::WN * OS + 16);
    return ring > rows ? ring : rows;
}

// BM x BN tiles, WM x WN waves, K tiles of BK in a ring of STAGES.  With KG
// groups of such waves each takes one run of the K tiles, in a ring of its
// own, and their sums meet in LDS at the end: where there are few output
// tiles this keeps more copies in flight a CU.
template <typename S, typename O>
__device__ __forceinline__ void mx_gemm_body(const MxGemmArgs &g, int id, unsigned char *smem)
{
    constexpr int BM = S::BM, BN = S::BN, BK = S::BK, WM = S::WM, NW = S::WM * S::WN, STAGES = S::STAGES, KG = S::KG;
    constexpr int TM = BM / S::WM, TN = BN / S::WN;         // a wave's tile
    constexpr int FM = TM / 32, FN = TN / 32;               // 32 x 32 blocks of a wave
    constexpr int ROWS = BM + BN;
    constexpr int C = BK / 32, Q = BK / 128, H = BK / 64;   // blocks, scale dwords and product steps of a K tile
    constexpr int CODES = S::CODES, STAGE = S::STAGE;
    constexpr int RPC = 64 / C;                             // rows a wave's copy
    constexpr int CP = ROWS / (NW * RPC);                   // code copies a wave and stage
    constexpr int SA = (BM + 63) / 64, SLOTS = S::SLOTS;    // slots of 64 rows' scale dwords: a's, then b's
    constexpr int SP = (SLOTS + NW - 1) / NW;               // scale copies (a slot each) a wave and dword
    constexpr int PER = CP + SP * Q;
    // Copies of a later tile that a K tile's last step issues, its first and
    // (the rest) its second: early enough to land, and spread, as each takes
    // several instructions (8192^3: 310 us with 8, 8 and 4 of 20, 313 with 10
    // and 10, 337 with all in the last step, 328 with none in it).
    constexpr int E0 = PER * 2 / 5, E1 = H > 2 ? PER * 2 / 5 : PER - E0;
    constexpr int OS = sizeof(typename O::raw);
    constexpr int PITCH = TN * OS + 16;                     // epilogue: 32 rows a wave
    static_assert((STAGES & (STAGES - 1)) == 0 && (STAGES - 2) * PER + E0 < 64, "ring of stages");
    static_assert(C == 4 || C == 8, "64 or 128 bytes a row");
    static_assert(BM % (NW * RPC) == 0 && BN % (NW * RPC) == 0,
                  "a pass of copies stays in one operand");

    const int lane = threadIdx.x & 63;
    const int thread = threadIdx.x % (NW * 64);
    const int wave = __builtin_amdgcn_readfirstlane(thread >> 6);
    const int group = KG > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / (NW * 64)) : 0;
    unsigned char *const lds = smem;
    smem += group * (STAGES * STAGE);
    const int wm = wave % WM, wn = wave / WM;
    const int half = lane >> 5, l32 = lane & 31;
    int tm, tn;
    mx_tile(g, id, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int quads = (g.kb + 3) / 4;
    // K tiles t0 .. t0 + nk - 1, blocks below kend; the groups run as many
    // steps each, the last ones on zeros
    const int nk = ((g.kb + C - 1) / C + KG - 1) / KG, t0 = group * nk;
    const int kend = KG > 1 ? min(g.kb, (t0 + nk) * C) : g.kb;

    const unsigned ca = (unsigned)g.M * g.kb * 16u, cb = (unsigned)g.N * g.kb * 16u;
    const unsigned na = (unsigned)g.M * quads * 4u, nb = (unsigned)g.N * quads * 4u;
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc((void *)g.a, 0, ca, kMxRsrcWord3);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc((void *)g.b, 0, cb, kMxRsrcWord3);

    // Copies of codes: this lane's row of each pass, and the physical 16-byte
    // chunk lane % C of that row.  Chunk c of row r lies at c ^ key(r): 16
    // rows' equal chunks then cover all banks.
    auto key = [](int r) { return C == 4 ? (r >> 2) & 3 : (r >> 1) & 7; };
    unsigned coff[CP];
    int cblk[CP];
#pragma unroll
    for (int p = 0; p < CP; ++p) {
        const int r = (p * NW + wave) * RPC + lane / C;
        const bool isa = p * NW * RPC < BM;
        const int row = isa ? m0 + r : n0 + r - BM;
        cblk[p] = (lane & (C - 1)) ^ key(r);
        coff[p] = row < (isa ? g.M : g.N) ? (unsigned)row * (unsigned)g.kb * 16u + cblk[p] * 16 : kMxOutOfRange;
    }
    // Copies of scales: a slot of 64 rows a wave instruction.
    __amdgpu_buffer_rsrc_t rs[SP];
    unsigned soff[SP], sstep[SP];
    int slot[SP];
#pragma unroll
    for (int p = 0; p < SP; ++p) {
        slot[p] = (p * NW + wave) % SLOTS;
        const bool isa = slot[p] < SA;
        const int row = isa ? m0 + slot[p] * 64 + lane : n0 + (slot[p] - SA) * 64 + lane;
        const int rows = isa ? g.M : g.N;
        rs[p] = __builtin_amdgcn_make_buffer_rsrc((void *)(isa ? g.sa : g.sb), 0, isa ? na : nb, kMxRsrcWord3);
        soff[p] = row < rows ? (unsigned)row * 4u : kMxOutOfRange;
        sstep[p] = (unsigned)rows * 4u;
    }
    // Copy c of K tile t into its stage.  Past the last block everything
    // reads as zeros, tiles past the last one included, so every stage counts
    // PER copies.
    auto issue1 = [&](int t, int c) {
        unsigned char *s = smem + (t & (STAGES - 1)) * STAGE;
        if (c < CP) {
            mx_dma16(c * NW * RPC < BM ? ra : rb, s + (c * NW + wave) * 1024,
                     t * C + cblk[c] < kend ? coff[c] + t * (C * 16u) : kMxOutOfRange);
        } else {
            const int p = (c - CP) / Q, q = (c - CP) % Q;
            mx_dma4(rs[p], s + CODES + (q * SLOTS + slot[p]) * 256, soff[p] + (t * Q + q) * sstep[p]);
        }
    };

    // The first K tile's copies, the bias (the sums start from it), the others'.
#pragma unroll
    for (int c = 0; c < PER; ++c)
        issue1(t0, c);
    f32x16_t acc[FM][FN];
    {
        const __amdgpu_buffer_rsrc_t rbias = __builtin_amdgcn_make_buffer_rsrc(
            (void *)g.bias, 0, g.bias && group == 0 ? (unsigned)g.N * 4u : 0u, kMxRsrcWord3);
        const int n = n0 + wn * TN + half * 4;
        if (n0 + BN <= g.N) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const u32v4_t v = __builtin_amdgcn_raw_buffer_load_b128(rbias, (n + j * 32 + q * 8) * 4u, 0, 0);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[0][j][4 * q + e] = __uint_as_float(v[e]);
                }
        } else {
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int c = n + j * 32 + (e >> 2) * 8 + (e & 3);
                    acc[0][j][e] = __uint_as_float(
                        __builtin_amdgcn_raw_buffer_load_b32(rbias, c < g.N ? c * 4u : kMxOutOfRange, 0, 0));
                }
        }
#pragma unroll
        for (int i = 1; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                acc[i][j] = acc[0][j];
    }
#pragma unroll
    for (int t = 1; t < STAGES; ++t)
#pragma unroll
        for (int c = 0; c < (t < STAGES - 1 ? PER : E0); ++c)
            issue1(t0 + t, c);

    // Step h of a K tile takes two blocks of each row.  Of eight, lanes 0 .. 31
    // take block h and the others block 4 + h, so that each half needs one
    // scale dword, byte h of it; of four, blocks 2 h and 2 h + 1 and byte 2 h,
    // the upper half's dword shifted down by a byte.
    const int arow = wm * TM + l32, brow = wn * TN + l32, k32 = key(l32);
    i32x4_t a[2][FM], b[2][FN];
    auto frag1 = [&](int t, int h, int k) {
        const int blk = C == 8 ? half * 4 + h : h * 2 + half;
        const unsigned char *s = smem + (t & (STAGES - 1)) * STAGE + ((blk ^ k32) * 16);
        if (k < FN)
            b[h & 1][k] = *(const i32x4_t *)(s + (BM + brow + k * 32) * (C * 16));
        else
            a[h & 1][k - FN] = *(const i32x4_t *)(s + (arow + (k - FN) * 32) * (C * 16));
    };
    unsigned wa[FM], wb[FN];
    auto scale1 = [&](int t, int k) {
        const unsigned char *s = smem + (t & (STAGES - 1)) * STAGE + CODES + (C == 8 ? half * (SLOTS * 256) : 0);
        if (k < FN)
            wb[k] = *(const unsigned *)(s + SA * 256 + (brow + k * 32) * 4);
        else
            wa[k - FN] = *(const unsigned *)(s + (arow + (k - FN) * 32) * 4);
    };

    // While the products of one step run, the next step's operands are read
    // and copies are issued, a few instructions in the shadow of each product
    // (32 cycles); the order is fixed here, as a run of reads or copies
    // without products between them leaves the matrix unit idle.  One barrier
    // a K tile, after the first product of its last step: tile t has been
    // read by then and tile t + 1 has landed; the copies of tile t + STAGES
    // follow it, the second half of them in the next step.
    constexpr int NM = FM * FN, FR = FM + FN;
    mx_wait_vm<(STAGES - 2) * PER + E0>();
    mx_barrier();
#pragma unroll
    for (int k = 0; k < FR; ++k) {
        frag1(t0, 0, k);
        scale1(t0, k);
    }
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    int t = t0;
    do {      // nk > 0
        int sa[FM], sb[FN];
        const int shift = C == 8 ? 0 : 8 * half;
#pragma unroll
        for (int i = 0; i < FM; ++i)
            sa[i] = (int)(wa[i] >> shift);
#pragma unroll
        for (int j = 0; j < FN; ++j)
            sb[j] = (int)(wb[j] >> shift);
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const bool last = h == H - 1;
            const int reads = last ? 2 * FR : FR;
            const int c0 = last ? 0 : h == 0 ? E0 : E0 + E1, copies = last ? E0 : h == 0 ? E1 : h == 1 ? PER - E0 - E1 : 0;
            const int pieces = reads + copies;
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                const int i = m / FN, j = m % FN;
                acc[i][j] = mx_mfma32(C == 8 ? h : 2 * h, b[h & 1][j], a[h & 1][i], acc[i][j], sb[j], sa[i]);
                if (last && m == 0) {
                    mx_wait_vm<(STAGES - 2) * PER>();
                    mx_wait_lds();
                    mx_barrier();
                }
#pragma unroll
                for (int k = m * pieces / NM; k < (m + 1) * pieces / NM; ++k) {
                    if (k < FR)
                        frag1(last ? t + 1 : t, last ? 0 : h + 1, k);
                    else if (k < reads)
                        scale1(t + 1, k - FR);
                    else
                        issue1(last ? t + STAGES : t + STAGES - 1, k - reads + c0);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        // (a fence: the compiler would sink the reads to the next iteration)
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
    } while (++t < t0 + nk);

    // Rows of the output through LDS, as many blocks of 32 a wave as it holds,
    // so that stores are 16 bytes a lane along the row.
    mx_wait_vm<0>();
    mx_wait_lds();
    mx_barrier();
    if constexpr (KG > 1) {
        // [block of 16 values][group - 1][the group's thread]
        f32x4_t *sums = (f32x4_t *)lds;
#pragma unroll
        for (int b = 0; b < FM * FN; ++b) {
            f32x16_t &v = acc[b / FN][b % FN];
            if (b > 0)
                mx_barrier();
            if (group > 0)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    sums[((group - 1) * 4 + q) * (NW * 64) + thread] =
                        f32x4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
            mx_wait_lds();
            mx_barrier();
            if (group == 0)
#pragma unroll
                for (int k = 0; k < KG - 1; ++k)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4_t u = sums[(k * 4 + q) * (NW * 64) + thread];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[4 * q + e] += u[e];
                    }
            mx_wait_lds();
        }
        mx_barrier();      // the sums have been read; the output's rows take their place
        if (group > 0)
            return;
    }
    constexpr int CHUNKS = TN * OS / 16, EPC = 16 / OS;      // 16-byte chunks a row, elements a chunk
    constexpr int RP = 64 / CHUNKS;                          // rows a wave instruction
    constexpr int FIT = STAGES * STAGE / (NW * 32 * PITCH), G = FIT < 1 ? 1 : FIT < FM ? FIT : FM;      // blocks at once
    static_assert(FM % G == 0 || G == 1, "whole groups");
#pragma unroll
    for (int i0 = 0; i0 < FM; i0 += G) {
#pragma unroll
        for (int i = 0; i < G; ++i) {
            unsigned char *mine = lds + (i * NW + wave) * 32 * PITCH;
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    unsigned char *p = mine + l32 * PITCH + (j * 32 + q * 8 + half * 4) * OS;
                    const float *v = (const float *)&acc[i0 + i][j] + q * 4;
                    if constexpr (OS == 4)
                        *(f32x4_t *)p = f32x4_t{v[0], v[1], v[2], v[3]};
                    else if constexpr (O::code == CONVIMG_BF16)
                        *(uint2 *)p = uint2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
                    else
                        *(uint2 *)p = uint2{pack_fp16(v[0], v[1]), pack_fp16(v[2], v[3])};
                }
        }
        mx_wait_lds();
        __builtin_amdgcn_wave_barrier();
        const int k = lane % CHUNKS, n = n0 + wn * TN + k * EPC;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const unsigned char *mine = lds + (i * NW + wave) * 32 * PITCH;
            const int m = m0 + wm * TM + (i0 + i) * 32, rows = min(g.M - m, 32);
            typename O::raw *o = (typename O::raw *)g.out + (long long)m * g.N + n;
            if (n + EPC <= g.N) {
#pragma unroll
                for (int p = 0; p < 32 / RP; ++p) {
                    const int r = p * RP + lane / CHUNKS;
                    const u32v4_t v = *(const u32v4_t *)(mine + r * PITCH + k * 16);
                    if (r < rows) {
                        if constexpr (OS == 4)
                            *(u32v4_a4_t *)(o + (long long)r * g.N) = v;
                        else
                            *(u32v4_a2_t *)(o + (long long)r * g.N) = v;
                    }
                }
            } else if (n < g.N) {
                for (int r = lane / CHUNKS; r < rows; r += RP)
                    for (int e = 0; n + e < g.N; ++e)
                        o[(long long)r * g.N + e] = ((const typename O::raw *)(mine + r * PITCH + k * 16))[e];
            }
        }
        if (i0 + G < FM) {
            mx_wait_lds();
            __builtin_amdgcn_wave_barrier();
        }
    }
}

template <typename S, typename O>
__global__ __launch_bounds__(S::threads) void mx_gemm_tile(MxGemmArgs g)
{
    __shared__ __attribute__((aligned(16))) unsigned char smem[mx_gemm_lds<S, sizeof(typename O::raw)>()];
    const unsigned id = mx_xcd_tile(blockIdx.x, gridDim.x);
    if (id < (unsigned)g.tm * g.tn)
        mx_gemm_body<S, O>(g, id, smem);
}

// Column sums from partial sums [parts][cols], 64 columns a workgroup.
struct MxSumArgs {
    const float *part;
    float *out;            // NULL: none
    int parts, cols;
};

__device__ __forceinline__ void mx_sum_parts(const MxSumArgs &a, unsigned block, float *lds)
{
    const int c = (int)block * 64 + (threadIdx.x & 63), w = threadIdx.x >> 6;
    float s = 0.f;
    if (c < a.cols)
#pragma unroll 4
        for (int p = w; p < a.parts; p += (int)blockDim.x / 64)
            s += a.part[(long long)p * a.cols + c];
    lds[threadIdx.x] = s;
    __syncthreads();
    if (w == 0 && c < a.cols) {
        s = 0.f;
        for (int k = threadIdx.x; k < (int)blockDim.x; k += 64)
            s += lds[k];
        a.out[c] = s;
    }
}

// Both products of the backward pass and the sums of db in one launch; the
// first `dw_blocks` workgroups take dw's tiles (fp32), the next `dx_blocks`
// those of dx, the others 64 columns of db each.
template <typename S, typename O>
__global__ __launch_bounds__(S::threads) void mx_gemm_bwd(MxGemmArgs dw, MxGemmArgs dx, MxSumArgs db,
                                                          unsigned dw_blocks, unsigned dx_blocks)
{
    __shared__ __attribute__((aligned(16))) unsigned char smem[mx_gemm_lds<S, 4>()];
    if (blockIdx.x < dw_blocks) {
        const unsigned id = mx_xcd_tile(blockIdx.x, dw_blocks);
        if (id < (unsigned)dw.tm * dw.tn)
            mx_gemm_body<S, Fp32>(dw, id, smem);
    } else if (blockIdx.x < dw_blocks + dx_blocks) {
        const unsigned id = mx_xcd_tile(blockIdx.x - dw_blocks, dx_blocks);
        if (id < (unsigned)dx.tm * dx.tn)
            mx_gemm_body<S, O>(dx, id, smem);
    } else {
        mx_sum_parts(db, blockIdx.x - dw_blocks - dx_blocks, (float *)smem);
    }
}

}  // namespace convimg
