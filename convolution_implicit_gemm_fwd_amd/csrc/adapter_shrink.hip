// adapter_shrink.hip -- h[m] = down_g x[m], g = ids[m], in one pass over x
// that also writes x's MXFP4 rows for the shared projection and, for training,
// its MXINT8 rows.
#include "adapter.hpp"

namespace convimg {

// ---- few rows --------------------------------------------------------------
//
// A workgroup takes kAdFewCols columns of one row, a thread eight of them, with
// its part of every rank's row of the adapter in flight at once: a serving batch
// mostly has another adapter in every row, whose 2 r K bytes are the work.  The
// parts' sums stay apart; what reads h adds them.
constexpr int kAdFewThreads = 128, kAdFewCols = kAdFewThreads * 8, kAdFewRanks = 16;

template <typename X, typename A>
__global__ __launch_bounds__(kAdFewThreads) void ad_shrink_few(AdShrinkArgs a)
{
    __shared__ float sums[2][kAdFewRanks];
    const int m = blockIdx.y, c = blockIdx.x * kAdFewCols + threadIdx.x * 8;
    const int id = a.ids[m];
    const bool has = id >= 0 && id < a.G;
    const Raw8<X> raw = load_raw8<X>((const typename X::raw *)a.x + m * a.ldx, c, a.K);
    float v[8];
    unpack8<X>(tail8<X>(raw, c, a.K), v);
    if (a.codes) {
        unsigned top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top = mx_top(top, v[e]);
        const unsigned byte = mx_scale_byte(quad_max(top));
        const int kb = mx_blocks(a.K);
        if (c < kb * 32)
            ((unsigned *)a.codes)[((long long)m * kb * 32 + c) / 8] = mx_encode8(v, mx_scale_value(byte));
        const unsigned word = mx_scale_word<16>(byte, c >> 5);
        if ((c & 127) == 0 && c < a.K)
            ((unsigned *)a.scales)[(long long)(c >> 7) * a.M + m] = word;
    }
    float *h = a.h + ((long long)blockIdx.x * a.M + m) * a.r;
    const typename A::raw *down = (const typename A::raw *)a.down + (long long)id * a.r * a.K;
    for (int i0 = 0; i0 < a.r; i0 += kAdFewRanks) {
        Raw8<A> w[kAdFewRanks];
        if (has)
#pragma unroll
            for (int i = 0; i < kAdFewRanks; ++i)
                w[i] = load_raw8<A>(down + (long long)min(i0 + i, a.r - 1) * a.K, c, a.K);
        __syncthreads();      // the previous sums have been read
#pragma unroll
        for (int i = 0; i < kAdFewRanks; ++i) {
            float s = 0.f;
            if (has) {
                float u[8];
                unpack8<A>(tail8<A>(w[i], c, a.K), u);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s = __builtin_fmaf(u[e], v[e], s);
            }
            s = group_sum<64>(s);
            if ((threadIdx.x & 63) == 0)
                sums[threadIdx.x >> 6][i] = s;
        }
        __syncthreads();
        if (threadIdx.x < kAdFewRanks && i0 + (int)threadIdx.x < a.r)
            h[i0 + threadIdx.x] = sums[0][threadIdx.x] + sums[1][threadIdx.x];
    }
}

// ---- many rows -------------------------------------------------------------
//
// A workgroup takes 16 rows, sorted by adapter, and 16 RT ranks; its eight waves
// share the columns in steps of 128.  Rows are loaded as they lie, 16 lanes a
// row, the next step in flight; in that form four lanes hold a block and quantise
// it.  They reach the matrix instruction's form (a lane eight columns of row
// lane % 16) through LDS that is the wave's own.  (Loading them in that form
// straight away puts neighbouring lanes on different rows: 8192 x 8192 71 us.)
// Where the 16 rows have several adapters, at the sorted runs' ends, x is read
// again (from cache) for each.
constexpr int kAdWaves = 8;

// 16 rows of 128 columns of a wave, in LDS.
template <typename T>
struct Strip16 {
    static constexpr int ES = sizeof(typename T::raw), PITCH = 128 * ES + 16, BYTES = 16 * PITCH;

    // lane l holds columns 8 (l % 16) .. of row 4 j + l / 16 in r[j]
    static __device__ __forceinline__ void put(unsigned char *lds, int lane, const Raw8<T> (&r)[4])
    {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *(Raw8<T> *)(lds + (4 * j + (lane >> 4)) * PITCH + (lane & 15) * 8 * ES) = r[j];
    }
    // columns 32 j + 8 (l / 16) .. of row l % 16
    static __device__ __forceinline__ Raw8<T> get(const unsigned char *lds, int lane, int j)
    {
        return *(const Raw8<T> *)(lds + (lane & 15) * PITCH + (j * 32 + (lane >> 4) * 8) * ES);
    }
};

// Eight columns from c on of a row that starts `off` bytes from base, zeros
// past its K; WHOLE: c + 8 <= K in every lane.
template <typename T, bool WHOLE>
__device__ __forceinline__ Raw8<T> strip_load(const char *base, unsigned off, int c, int K)
{
    constexpr int ES = sizeof(typename T::raw);
    if constexpr (WHOLE) {
        Raw8<T> r;
        const char *p = base + (off + (unsigned)c * ES);
        if constexpr (ES == 4) {
            r.w[0] = ((const u32v4_a4_t *)p)[0];
            r.w[1] = ((const u32v4_a4_t *)p)[1];
        } else {
            r.w[0] = *(const u32v4_a2_t *)p;
        }
        return r;
    } else {
        return tail8<T>(load_raw8<T>((const typename T::raw *)(base + off), c, K), c, K);
    }
}

template <typename X, typename A, int RT>
__global__ __launch_bounds__(kAdWaves * 64) void ad_shrink_tile(AdShrinkArgs a)
{
    constexpr int LDS = kAdWaves * (Strip16<X>::BYTES + Strip16<A>::BYTES), SUMS = kAdWaves * RT * 64 * 16;
    __shared__ __attribute__((aligned(16))) unsigned char lds[LDS > SUMS ? LDS : SUMS];
    const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = blockIdx.x * 16, i0 = blockIdx.y * 16 * RT;
    const int kb = mx_blocks(a.K), quads = (a.K + 127) / 128, end = quads * 128;
    unsigned char *const xs = lds + wave * Strip16<X>::BYTES,
                  *const ws = lds + kAdWaves * Strip16<X>::BYTES + wave * Strip16<A>::BYTES;
    f32x4_t(*sums)[RT][64] = (f32x4_t(*)[RT][64])lds;

    // row r16 and the rows 4 j + q, the last one again past the end
    const bool real = m0 + r16 < a.M;
    const int at = min(m0 + r16, a.M - 1), m = a.order ? a.order[at] : at;
    const int given = real ? a.ids[m] : -1, id = given < a.G ? given : -1;
    unsigned left = (unsigned)__ballot(id >= 0) & 0xffffu;
    const char *x[4];
    int xrow[4];
    unsigned woff[4];      // rank 4 j + q of a tile of ranks; a tile that would pass the rank ends with it
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        xrow[j] = __shfl(m, 4 * j + q);
        x[j] = (const char *)a.x + (long long)xrow[j] * a.ldx * (long long)sizeof(typename X::raw);
        woff[j] = (unsigned)min(4 * j + q, a.r - 1) * (unsigned)a.K * (unsigned)sizeof(typename A::raw);
    }
    if (real && id < 0)      // no adapter: 0
        for (int i = i0 + (threadIdx.x >> 4); i < min(a.r, i0 + 16 * RT); i += kAdWaves * 4) {
            a.h[(long long)at * a.r + i] = 0.f;
            if (a.kept)
                a.kept[(long long)m * a.r + i] = 0.f;
        }

    bool first = blockIdx.y == 0;
    do {
        int g = -1;
        if (left) {
            g = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
            left &= ~(unsigned)__ballot(id == g);
        }
        if (!first && g < 0)
            return;      // (a further chunk of ranks for rows without adapters)
        f32x4_t acc[RT] = {};
        Raw8<X> xn[4];      // the next step's
        Raw8<A> wn[4];      // 16 ranks, the next ones'
        auto fetch = [&](int k0) {
            const int c = k0 + r16 * 8;
            if (k0 + 128 <= a.K) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    xn[j] = strip_load<X, true>(x[j], 0, c, a.K);
            } else if (k0 < end) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    xn[j] = strip_load<X, false>(x[j], 0, c, a.K);
            }
        };
        auto fetch_w = [&](int t, int k0) {
            const int c = k0 + r16 * 8, row = min(i0 + t * 16, max(a.r - 16, 0));
            const char *w =
                (const char *)a.down + ((long long)max(g, 0) * a.r + row) * a.K * (long long)sizeof(typename A::raw);
            if (k0 + 128 <= a.K) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    wn[j] = strip_load<A, true>(w, woff[j], c, a.K);
            } else if (k0 < end) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    wn[j] = strip_load<A, false>(w, woff[j], c, a.K);
            }
        };
        fetch(wave * 128);
        fetch_w(0, wave * 128);
        for (int k0 = wave * 128; k0 < end; k0 += kAdWaves * 128) {
            const int c = k0 + r16 * 8;
            Raw8<X> xr[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                xr[j] = xn[j];
            Strip16<X>::put(xs, lane, xr);
            fetch(k0 + kAdWaves * 128);
            if (first && (a.codes || a.codes8)) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int p = m0 + 4 * j + q;
                    const bool on = p < a.M;
                    float v[8];
                    unpack8<X>(xr[j], v);
                    unsigned top = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        top = mx_top(top, v[e]);
                    top = quad_max(top);
                    if (a.codes) {
                        const unsigned byte = mx_scale_byte(top);
                        if (on && c < kb * 32)
                            *(unsigned *)(a.codes + ((long long)(m0 + 4 * j) * (kb * 16) + (unsigned)(q * (kb * 16) + c / 2))) =
                                mx_encode8(v, mx_scale_value(byte));
                        const unsigned word = mx_scale_word<16>(byte, c >> 5);
                        if (on && r16 == 0)
                            ((unsigned *)a.scales)[(long long)(k0 >> 7) * a.M + p] = word;
                    }
                    if (a.codes8) {
                        const unsigned byte = mxi_scale_byte(top);
                        if (on && c < kb * 32)
                            *(uint2 *)(a.codes8 + ((long long)xrow[j] * (kb * 32) + c)) = mxi_encode8(v, byte);
                        const unsigned word = mx_scale_word<16>(c < kb * 32 ? byte : 0u, c >> 5);
                        if (on && r16 == 0)
                            ((unsigned *)a.scales8)[(long long)xrow[j] * quads + (k0 >> 7)] = word;
                    }
                }
            }
            if (g < 0)
                continue;
            u32v4_t xf[4][split_terms<X>()];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                split_raw8<X>(Strip16<X>::get(xs, lane, j), xf[j]);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                Strip16<A>::put(ws, lane, wn);
                fetch_w(t + 1 < RT ? t + 1 : 0, t + 1 < RT ? k0 : k0 + kAdWaves * 128);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    u32v4_t wf[split_terms<A>()];
                    split_raw8<A>(Strip16<A>::get(ws, lane, j), wf);
                    acc[t] = mfma_terms16(wf, xf[j], acc[t]);
                }
            }
        }
        first = false;
        if (g < 0)
            break;
        // the waves' sums in order; a lane holds ranks 4 q .. 4 q + 3 of row r16
        __syncthreads();
#pragma unroll
        for (int t = 0; t < RT; ++t)
            sums[wave][t][lane] = acc[t];
        __syncthreads();
        if (wave < RT) {
            f32x4_t s = sums[0][wave][lane];
#pragma unroll
            for (int w = 1; w < kAdWaves; ++w)
                s += sums[w][wave][lane];
            const int want = i0 + wave * 16, row = min(want, max(a.r - 16, 0));
            if (id == g)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = row + q * 4 + e;
                    if (i >= want && i < a.r) {
                        a.h[(long long)at * a.r + i] = s[e];
                        if (a.kept)
                            a.kept[(long long)m * a.r + i] = s[e];
                    }
                }
        }
        __syncthreads();
    } while (left);
}

// ---- the rows sorted by adapter --------------------------------------------
//
// By one workgroup, eight bits of the adapter's number at a time (once for up
// to 255 adapters), stably: each wave counts the digits of its run of rows, the
// counts become places, and a row's place is its wave's next one for the digit
// plus the number of equal digits in lower lanes.
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;

__global__ __launch_bounds__(kSortThreads) void ad_sort(const int *ids, int M, int G, int bits, int *order, int *temp,
                                                        int *start)
{
    __shared__ int place[256][kSortWaves];
    __shared__ int waves[kSortWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int run = (int)((M + kSortWaves * 64LL - 1) / (kSortWaves * 64)) * 64;
    const long long lo = (long long)wave * run;
    const int hi = (int)min((long long)M, lo + run);
    auto key_of = [&](int row) {
        const int k = ids[row];
        return k < 0 || k > G ? G : k;
    };
    // (the last pass writes `order`)
    int *out = (bits + 7) / 8 % 2 ? order : temp;
    const int *in = nullptr;
    for (int shift = 0; shift < bits; shift += 8) {
        for (int k = threadIdx.x; k < 256 * kSortWaves; k += kSortThreads)
            (&place[0][0])[k] = 0;
        __syncthreads();
        for (long long p = lo + lane; p < hi; p += 64)
            atomicAdd(&place[(key_of(in ? in[p] : (int)p) >> shift) & 255][wave], 1);
        __syncthreads();
        // counts to places: thread t holds four waves of digit t / 4
        int *mine = &place[0][0] + threadIdx.x * 4, sum = mine[0] + mine[1] + mine[2] + mine[3], upto = sum;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(upto, o);
            upto += lane >= o ? v : 0;
        }
        if (lane == 63)
            waves[wave] = upto;
        __syncthreads();
        int before = upto - sum;
        for (int w = 0; w < wave; ++w)
            before += waves[w];
        for (int k = 0; k < 4; ++k) {
            const int n = mine[k];
            mine[k] = before;
            before += n;
        }
        __syncthreads();
        if (start && bits <= 8)
            for (int g = threadIdx.x; g <= G; g += kSortThreads)
                start[g] = place[g][0];
        __syncthreads();
        for (long long p0 = lo; p0 < hi; p0 += 64) {
            const long long p = p0 + lane;
            const bool on = p < hi;
            const int row = on ? (in ? in[p] : (int)p) : 0;
            const unsigned digit = on ? (key_of(row) >> shift) & 255 : 0;
            unsigned long long same = __ballot(on);
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                const unsigned long long set = __ballot(digit >> b & 1);
                same &= digit >> b & 1 ? set : ~set;
            }
            const int rank = __builtin_amdgcn_mbcnt_hi((unsigned)(same >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)same, 0));
            if (on) {
                const int at = place[digit][wave];
                out[at + rank] = row;
                if (rank == 0)
                    place[digit][wave] = at + __builtin_popcountll(same);
            }
        }
        __threadfence_block();
        __syncthreads();
        in = out;
        out = out == order ? temp : order;
    }
    if (start && bits > 8)
        for (int g = threadIdx.x; g <= G; g += kSortThreads) {
            int a = 0, b = M;      // the first place whose adapter is at least g
            while (a < b) {
                const int mid = a + (b - a) / 2;
                if (key_of(order[mid]) < g)
                    a = mid + 1;
                else
                    b = mid;
            }
            start[g] = a;
        }
}

void adapter_sort(const int *ids, int M, int G, int *order, int *start, hipStream_t stream)
{
    int bits = 1;
    while (bits < 32 && (unsigned)G >> bits)
        ++bits;
    hipLaunchKernelGGL(ad_sort, dim3(1), dim3(kSortThreads), 0, stream, ids, M, G, bits, order, order + M, start);
}

// A row a workgroup for up to 64 rows, and for up to 1024 where the adapters
// may be so many that the rows hardly share any.
AdPlan adapter_plan(int M, int K, int G, bool keep)
{
    AdPlan p;
    p.few = !keep && (M <= 64 || (M <= 1024 && M < 8LL * G));
    p.sorted = !p.few && G > 1;
    p.splits = p.few ? (K + kAdFewCols - 1) / kAdFewCols : 1;
    return p;
}

void adapter_shrink(const AdShrinkArgs &a, const AdPlan &plan, int x_dtype, int a_dtype, hipStream_t stream)
{
    with_dtype(x_dtype, [&](auto x) {
        with_dtype(a_dtype, [&](auto w) {
            typedef decltype(x) X;
            typedef decltype(w) A;
            if (plan.few) {
                hipLaunchKernelGGL((ad_shrink_few<X, A>), dim3(plan.splits, a.M), dim3(kAdFewThreads), 0, stream, a);
                return;
            }
            const unsigned tiles = (unsigned)((a.M + 15LL) / 16);
            if (a.r <= 16)
                hipLaunchKernelGGL((ad_shrink_tile<X, A, 1>), dim3(tiles), dim3(kAdWaves * 64), 0, stream, a);
            else if (a.r <= 32)
                hipLaunchKernelGGL((ad_shrink_tile<X, A, 2>), dim3(tiles), dim3(kAdWaves * 64), 0, stream, a);
            else
                hipLaunchKernelGGL((ad_shrink_tile<X, A, 4>), dim3(tiles, (a.r + 63) / 64), dim3(kAdWaves * 64), 0,
                                   stream, a);
        });
    });
}

}  // namespace convimg
