// adapter_shrink.hip -- h[m] = down_g x[m], g = ids[m], in one pass over x
// that also writes x's MXFP4 rows for the shared projection and, for training,
// its MXINT8 rows.
#include "adapter.hpp"

namespace convimg {

// h of one rank of a place, with its terms for the products.
__device__ __forceinline__ void adapter_put(const AdShrinkArgs &a, int at, int row, int i, float h, float scale)
{
    const int rp = adapter_ranks(a.r);
    a.h[(long long)at * rp + i] = h;
    if (a.kept && i < a.r)
        a.kept[(long long)row * a.r + i] = h;
    if (a.terms) {
        unsigned short t[3];
        adapter_terms(h * scale, t);
        unsigned short *p = (unsigned short *)(a.terms + ((long long)at * (rp / 16) + i / 16) * kAdTermBytes) + i % 16;
#pragma unroll
        for (int k = 0; k < 3; ++k)
            p[k * 16] = t[k];
    }
}

// ---- few rows --------------------------------------------------------------
//
// A workgroup takes four ranks of one row, a thread eight of every 4096 columns,
// with its part of each rank's row of the adapter in flight at once: a serving
// batch mostly has another adapter in every row, whose 2 r K bytes are the work.
// The latency of one read bounds it: 3.1 us for one row of 4096 columns and 16
// ranks, 3.4 for 64 rows with 64 adapters.  (16 ranks a workgroup read x fewer
// times, but their sums across the wave take longer: 6.5 and 7.2 us, and 10
// against 8.3 for 256 rows.)
constexpr int kAdFewWaves = 8, kAdFewRanks = 4;

template <typename X, typename A>
__global__ __launch_bounds__(kAdFewWaves * 64) void ad_shrink_few(AdShrinkArgs a)
{
    constexpr int RC = kAdFewRanks;
    __shared__ float sums[kAdFewWaves][RC];
    const int m = blockIdx.x, i0 = blockIdx.y * RC, wave = threadIdx.x >> 6;
    const int id = a.key[m];
    const bool has = id >= 0 && id < a.G;
    const typename X::raw *x = (const typename X::raw *)a.x + m * a.ldx;
    const typename A::raw *down = (const typename A::raw *)a.down + (long long)id * a.r * a.K;
    float s[RC] = {};
    const int end = (a.K + 127) & ~127;      // (the lanes of a scale dword stay together)
    for (int c = threadIdx.x * 8; c < end; c += kAdFewWaves * 512) {
        const Raw8<X> raw = load_raw8<X>(x, c, a.K);
        Raw8<A> w[RC];
        if (has)
#pragma unroll
            for (int i = 0; i < RC; ++i)
                w[i] = load_raw8<A>(down + (long long)min(i0 + i, a.r - 1) * a.K, c, a.K);
        float v[8];
        unpack8<X>(tail8<X>(raw, c, a.K), v);
        if (blockIdx.y == 0 && (a.codes || a.codes8)) {
            unsigned top = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                top = mx_top(top, v[e]);
            if (a.codes) {
                const unsigned byte = mx_scale_byte(quad_max(top));
                const int kb = mx_blocks(a.K);
                if (c < kb * 32)
                    ((unsigned *)a.codes)[((long long)m * kb * 32 + c) / 8] = mx_encode8(v, mx_scale_value(byte));
                const unsigned word = mx_scale_word<16>(byte, c >> 5);
                if ((c & 127) == 0)
                    ((unsigned *)a.scales)[(long long)(c >> 7) * a.M + m] = word;
            }
            if (a.codes8)
                mxi_emit8<16>(a.codes8, (unsigned *)a.scales8, m, a.K, c, v);
        }
        if (has)
#pragma unroll
            for (int i = 0; i < RC; ++i) {
                float u[8];
                unpack8<A>(tail8<A>(w[i], c, a.K), u);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s[i] = __builtin_fmaf(u[e], v[e], s[i]);
            }
    }
#pragma unroll
    for (int i = 0; i < RC; ++i) {
        const float t = group_sum<64>(s[i]);
        if ((threadIdx.x & 63) == 0)
            sums[wave][i] = t;
    }
    __syncthreads();
    const int i = i0 + (int)threadIdx.x;
    if (threadIdx.x < RC && i < adapter_ranks(a.r)) {
        float h = 0.f;
        for (int k = 0; k < kAdFewWaves; ++k)
            h += sums[k][threadIdx.x];
        adapter_put(a, m, m, i, has && i < a.r ? h : 0.f, has ? a.scale[id] : 0.f);
    }
}

// ---- many rows -------------------------------------------------------------
//
// A workgroup takes 16 rows, sorted by adapter, and 16 RT ranks; its eight waves
// share the columns in steps of 128.  Rows are loaded as they lie, 16 lanes a
// row, the next step in flight; in that form four lanes hold a block and quantise
// it.  They reach the matrix instruction's form (a lane eight columns of row
// lane % 16) through LDS that is the wave's own.  (Loading them in that form
// straight away puts neighbouring lanes on different rows: 8192 x 8192 71 us, x
// in cache, against 40.  Two steps in flight overflow the registers: 2011 x 4096 with 64
// ranks 28 us against 19.)
//
// 8192 x 8192 and 16 ranks, x from memory: 51 us, 144 MB read and 37 written, 3.5
// TB/s (quantising alone 42 us there); 8192 x 4096 30 us.  The steps wait for their
// loads, and few of them are in flight: of 213 to 256 registers a lane (by the
// types and RT) a SIMD holds two waves, so a CU one workgroup of eight.  fp32 rows
// spill 84 to 284 bytes a lane, fp16 or bf16 rows with 64 ranks of another type up
// to 152.  (Held to four waves a SIMD all spill and take twice as long.)
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
    // what lane l put
    static __device__ __forceinline__ Raw8<T> own(const unsigned char *lds, int lane, int j)
    {
        return *(const Raw8<T> *)(lds + (4 * j + (lane >> 4)) * PITCH + (lane & 15) * 8 * ES);
    }
    // A strip that the rows' end cuts: value by value, zeros past it.  `row`
    // gives the address of row r, which lane r holds.
    static __device__ __forceinline__ void fill(unsigned char *lds, int lane, const char *row, int k0, int K)
    {
        // (loads at clamped places, 16 in flight)
#pragma unroll 1
        for (int e0 = lane; e0 < 16 * 128; e0 += 16 * 64) {
            typename T::raw v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int e = e0 + i * 64;
                const typename T::raw *p = (const typename T::raw *)__shfl((unsigned long long)row, e >> 7);
                v[i] = p[min(k0 + (e & 127), K - 1)];
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int e = e0 + i * 64;
                *(typename T::raw *)(lds + (e >> 7) * PITCH + (e & 127) * ES) =
                    k0 + (e & 127) < K ? v[i] : (typename T::raw)0;
            }
        }
    }
    // columns c .. c + 7 of a row
    static __device__ __forceinline__ Raw8<T> load(const char *row, unsigned c)
    {
        Raw8<T> r;
        const char *p = row + c * ES;
        if constexpr (ES == 4) {
            r.w[0] = ((const u32v4_a4_t *)p)[0];
            r.w[1] = ((const u32v4_a4_t *)p)[1];
        } else {
            r.w[0] = *(const u32v4_a2_t *)p;
        }
        return r;
    }
    // columns 32 j + 8 (l / 16) .. of row l % 16
    static __device__ __forceinline__ Raw8<T> get(const unsigned char *lds, int lane, int j)
    {
        return *(const Raw8<T> *)(lds + (lane & 15) * PITCH + (j * 32 + (lane >> 4) * 8) * ES);
    }
};

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

template <typename X, typename A, int RT>
__global__ __launch_bounds__(kAdWaves * 64) void ad_shrink_tile(AdShrinkArgs a)
{
    // (both fp16: their own instruction, which has the exact products, too)
    constexpr bool HALVES = __is_same(X, Fp16) && __is_same(A, Fp16);
    constexpr int LDS = kAdWaves * (Strip16<X>::BYTES + Strip16<A>::BYTES), SUMS = kAdWaves * RT * 64 * 16;
    __shared__ __attribute__((aligned(16))) unsigned char lds[LDS > SUMS ? LDS : SUMS];
    const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i0 = blockIdx.y * 16 * RT, rp = adapter_ranks(a.r);
    const int kb = mx_blocks(a.K), quads = (a.K + 127) / 128, end = quads * 128;
    unsigned char *const xs = lds + wave * Strip16<X>::BYTES,
                  *const ws = lds + kAdWaves * Strip16<X>::BYTES + wave * Strip16<A>::BYTES;
    f32x4_t(*sums)[RT][64] = (f32x4_t(*)[RT][64])lds;
    unsigned woff[4];      // rank 4 j + q of a tile of ranks; a tile that would pass the rank ends with it
#pragma unroll
    for (int j = 0; j < 4; ++j)
        woff[j] = (unsigned)min(4 * j + q, a.r - 1) * (unsigned)a.K * (unsigned)sizeof(typename A::raw);

    // A tile's own workgroup quantises its rows and takes the adapter that they
    // begin with (or have, unsorted); of an adapter that begins inside a tile one
    // of the workgroups behind the tiles' takes care.
    const int tiles = (int)((a.M + 15LL) / 16);
    const bool own = (int)blockIdx.x < tiles;
    for (int turn = (int)blockIdx.x - tiles; own || turn < a.G; turn += (int)gridDim.x - tiles) {
        int m0 = (int)blockIdx.x * 16;
        if (!own) {
            const int s = a.start[turn];
            if (s == a.start[turn + 1] || (s & 15) == 0)
                continue;
            m0 = s & ~15;
        }
        // row r16 and the rows 4 j + q, the last one again past the end
        const bool real = m0 + r16 < a.M;
        const int at = min(m0 + r16, a.M - 1), m = a.order ? a.order[at] : at;
        const int given = real ? a.key[at] : -1, id = given < a.G ? given : -1;
        const unsigned have = (unsigned)__ballot(id >= 0) & 0xffffu;
        const int g = own ? (have ? __builtin_amdgcn_readlane(id, __builtin_ctz(have)) : -1) : turn;
        const char *x[4];
        int xrow[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            xrow[j] = __shfl(m, 4 * j + q);
            x[j] = (const char *)a.x + (long long)xrow[j] * a.ldx * (long long)sizeof(typename X::raw);
        }
        if (own && real && id < 0)      // no adapter: 0
            for (int i = i0 + (threadIdx.x >> 4); i < min(rp, i0 + 16 * RT); i += kAdWaves * 4)
                adapter_put(a, at, m, i, 0.f, 0.f);
        const bool quantise = own && blockIdx.y == 0 && (a.codes || a.codes8);
        if (g < 0 && !quantise)
            return;
        f32x4_t acc[RT] = {};
        Raw8<X> xn[4];      // the next step's
        Raw8<A> wn[4];      // the next 16 ranks'
        // Each workgroup starts at another place of the columns: rows a power of
        // two apart would otherwise all be read from the same memory channels.
        const int span = kAdWaves * 128, laps = (end + span - 1) / span;
        const int begin = (int)(blockIdx.x % (unsigned)laps) * span + wave * 128;
        auto strip = [&](int lap) {      // past the last lap the end
            const int k = begin + lap * span;
            return lap >= laps ? end : k >= laps * span ? k - laps * span : k;
        };
        auto fetch = [&](int k0) {
            if (k0 + 128 <= a.K)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    xn[j] = Strip16<X>::load(x[j], (unsigned)(k0 + r16 * 8));
        };
        // 16 ranks of the adapter from its tile t on
        auto ranks = [&](int t) {
            return (const char *)a.down + ((long long)max(g, 0) * a.r + min(i0 + t * 16, max(a.r - 16, 0))) * a.K
                   * (long long)sizeof(typename A::raw);
        };
        auto fetch_w = [&](int t, int k0) {
            if (k0 + 128 <= a.K) {
                const char *w = ranks(t);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    wn[j] = Strip16<A>::load(w + woff[j], (unsigned)(k0 + r16 * 8));
            }
        };
        fetch(strip(0));
        fetch_w(0, strip(0));
        for (int lap = 0; lap < laps; ++lap) {
            const int k0 = strip(lap), c = k0 + r16 * 8;
            const bool inside = k0 + 128 <= a.K, some = k0 < end;
            Raw8<X> xr[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                xr[j] = xn[j];
            if (inside) {
                Strip16<X>::put(xs, lane, xr);
            } else if (some) {
                Strip16<X>::fill(xs, lane, (const char *)a.x + (long long)m * a.ldx * (long long)sizeof(typename X::raw), k0,
                                 a.K);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    xr[j] = Strip16<X>::own(xs, lane, j);
            }
            fetch(strip(lap + 1));
            // (all four rows of a lane side by side: one after another, each
            // step waits for the one before; 8192 x 8192 48 us, x in cache, against 40)
            if (some && quantise)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int p = m0 + 4 * j + q, row = xrow[j];
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
                            *(unsigned *)(a.codes + ((long long)p * (kb * 16) + c / 2)) = mx_encode8(v, mx_scale_value(byte));
                        const unsigned word = mx_scale_word<16>(byte, c >> 5);
                        if (on && r16 == 0)
                            ((unsigned *)a.scales)[(long long)(k0 >> 7) * a.M + p] = word;
                    }
                    if (a.codes8) {
                        const unsigned byte = mxi_scale_byte(top);
                        if (on && c < kb * 32)
                            *(uint2 *)(a.codes8 + ((long long)row * (kb * 32) + c)) = mxi_encode8(v, byte);
                        const unsigned word = mx_scale_word<16>(c < kb * 32 ? byte : 0u, c >> 5);
                        if (on && r16 == 0)
                            ((unsigned *)a.scales8)[(long long)row * quads + (k0 >> 7)] = word;
                    }
                }
            if (g < 0)
                continue;
            u32v4_t xf[4][HALVES ? 1 : split_terms<X>()];
            if (some)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const Raw8<X> r = Strip16<X>::get(xs, lane, j);
                    if constexpr (HALVES)
                        xf[j][0] = r.w[0];
                    else
                        split_raw8<X>(r, xf[j]);
                }
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                if (inside)
                    Strip16<A>::put(ws, lane, wn);
                else if (some)
                    Strip16<A>::fill(ws, lane,
                                     ranks(t) + (long long)min(r16, a.r - 1) * a.K * (long long)sizeof(typename A::raw), k0,
                                     a.K);
                fetch_w((t + 1) % RT, strip(lap + (t + 1) / RT));
                if (some)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const Raw8<A> r = Strip16<A>::get(ws, lane, j);
                        if constexpr (HALVES) {
                            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, r.w[0]),
                                                                            __builtin_bit_cast(f16x8_t, xf[j][0]), acc[t], 0,
                                                                            0, 0);
                        } else {
                            u32v4_t wf[split_terms<A>()];
                            split_raw8<A>(r, wf);
                            acc[t] = mfma_terms16(wf, xf[j], acc[t]);
                        }
                    }
            }
        }
        if (g < 0)
            return;
        // the waves' sums in order; a lane holds ranks 4 q .. 4 q + 3 of row r16
        __syncthreads();
#pragma unroll
        for (int t = 0; t < RT; ++t)
            sums[wave][t][lane] = acc[t];
        // An infinity times a lower term, which may be 0, made NaN: such a sum over
        // the wave's columns once more, value by value.
        if constexpr (!HALVES && split_terms<X>() + split_terms<A>() > 2) {
            bool nan = false;
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    nan |= acc[t][e] != acc[t][e];
            if (nan && id == g) {
                // (through empty asm: nothing of this is computed, and held in registers,
                // before it is known to be wanted)
                int K = a.K, row = m, four = 4 * q, adapter = g, r0 = i0;
                asm volatile("" : "+s"(K), "+v"(row), "+v"(four), "+v"(adapter), "+s"(r0));
#pragma unroll 1
                for (int k = 0; k < RT * 4; ++k) {
                    float &sum = ((float *)&sums[wave][k / 4][lane])[k % 4];
                    if (sum == sum)
                        continue;
                    const typename X::raw *x1 = (const typename X::raw *)a.x + row * a.ldx;
                    const typename A::raw *w = (const typename A::raw *)a.down
                        + ((long long)adapter * a.r + min(min(r0 + k / 4 * 16, max(a.r - 16, 0)) + four + k % 4, a.r - 1)) * K;
                    float s = 0.f;
#pragma unroll 1
                    for (int lap = 0; lap < laps && s == s; ++lap)
#pragma unroll 1
                        for (int c = strip(lap), last = min(c + 128, K); c < last && s == s; c += 8) {
                            float v[8], u[8];
                            load8<X>(x1, c, K, v);
                            load8<A>(w, c, K, u);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                s = __builtin_fmaf(u[e], v[e], s);
                        }
                    sum = s;
                }
            }
        }
        __syncthreads();
        if (wave < RT) {
            f32x4_t s = sums[0][wave][lane];
#pragma unroll
            for (int w = 1; w < kAdWaves; ++w)
                s += sums[w][wave][lane];
            const float scale = a.scale[g];
            const int want = i0 + wave * 16, row = min(want, max(a.r - 16, 0));
            if (id == g)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = row + q * 4 + e, past = want + q * 4 + e;
                    if (past >= a.r && past < rp)
                        adapter_put(a, at, m, past, 0.f, 0.f);
                    if (i >= want && i < a.r)
                        adapter_put(a, at, m, i, s[e], scale);
                }
        }
        if (own)
            return;
        __syncthreads();
    }
}

// ---- the rows sorted by adapter --------------------------------------------
//
// By one workgroup, eight bits of the adapter's number at a time (once for up
// to 255 adapters), stably, 512 rows of a wave in flight: each wave counts the
// digits of its run of rows, the counts become places, and a row's place is its
// wave's next one for the digit plus the number of equal digits in lower lanes.
// Lanes with equal digits find each other by a ballot for each bit in use, and
// one of them counts for all (an LDS atomic a lane: equal ones wait for each
// other, 16 us for 8192 rows of 4 adapters against 10; 2011 rows 5 us, 200 3.6).
// It is latency all along; several workgroups would have to wait for each other.
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;

__global__ __launch_bounds__(kSortThreads) void ad_sort(const int *ids, int M, int G, int bits, int *order, int *temp,
                                                        int *key, int *start, int *nan)
{
    if (nan && threadIdx.x == 0)
        *nan = 0;
    constexpr int U = 8;      // chunks of 64 rows in flight
    __shared__ int place[256][kSortWaves];
    __shared__ int waves[kSortWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int run = (int)((M + kSortWaves * 64LL - 1) / (kSortWaves * 64)) * 64;
    const long long lo = (long long)wave * run, hi = min((long long)M, lo + run);
    // (the last pass writes `order`)
    int *out = (bits + 7) / 8 % 2 ? order : temp;
    const int *in = nullptr;
    int row[U], kk[U];
    auto load = [&](long long p0) {      // rows and keys of U chunks, -1 past the run
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long p = p0 + u * 64 + lane;
            row[u] = p < hi ? (in ? in[p] : (int)p) : -1;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = row[u] >= 0 ? ids[row[u]] : 0;
            kk[u] = k < 0 || k > G ? G : k;
        }
    };
    // the lanes with the same digit
    auto matching = [&](bool on, unsigned digit, int n) {
        unsigned long long same = __ballot(on);
        for (int b = 0; b < n; ++b) {
            const unsigned long long set = __ballot(digit >> b & 1);
            same &= digit >> b & 1 ? set : ~set;
        }
        return same;
    };
    for (int shift = 0; shift < bits; shift += 8) {
        auto digit_of = [&](int u) { return row[u] >= 0 ? (unsigned)kk[u] >> shift & 255 : 0u; };
        if (lo < hi)
            load(lo);
        for (int k = threadIdx.x; k < 256 * kSortWaves; k += kSortThreads)
            (&place[0][0])[k] = 0;
        __syncthreads();
        for (long long p0 = lo; p0 < hi; p0 += U * 64) {
            if (p0 > lo)
                load(p0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (p0 + u * 64 >= hi)
                    break;
                const unsigned long long same = matching(row[u] >= 0, digit_of(u), min(bits - shift, 8));
                if (row[u] >= 0 && lane == __builtin_ctzll(same))
                    place[digit_of(u)][wave] += __builtin_popcountll(same);
            }
        }
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
        for (long long p0 = lo; p0 < hi; p0 += U * 64) {
            if (run > U * 64)      // (else the rows are still there)
                load(p0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (p0 + u * 64 >= hi)
                    break;
                const bool on = row[u] >= 0;
                const unsigned digit = digit_of(u);
                const unsigned long long same = matching(on, digit, min(bits - shift, 8));
                const int rank =
                    __builtin_amdgcn_mbcnt_hi((unsigned)(same >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)same, 0));
                if (on) {
                    const int at = place[digit][wave];
                    out[at + rank] = row[u];
                    if (shift + 8 >= bits)
                        key[at + rank] = kk[u] < G ? kk[u] : -1;
                    if (rank == 0)
                        place[digit][wave] = at + __builtin_popcountll(same);
                }
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
                const int mid = a + (b - a) / 2, k = key[mid];
                if ((k < 0 ? G : k) < g)
                    a = mid + 1;
                else
                    b = mid;
            }
            start[g] = a;
        }
}

void adapter_sort(const int *ids, int M, int G, int *order, int *key, int *start, int *nan, hipStream_t stream)
{
    int bits = 1;
    while (bits < 32 && (unsigned)G >> bits)
        ++bits;
    hipLaunchKernelGGL(ad_sort, dim3(1), dim3(kSortThreads), 0, stream, ids, M, G, bits, order, order + M, key,
                       start, nan);
}

// A row a workgroup for up to 256 rows, unsorted; 16 sorted rows a workgroup
// above.  With 4096 x 4096 and 16 ranks, sorting and the product included: 64
// rows of 4 adapters 12 us against 22 sorted, 256 rows of 8 adapters 18.5 against
// 24.5 and of 32 24.4 against 25.6, 512 rows of 16 adapters 29.5 against 29.  Each
// row reads its adapter for itself, so more ranks move the bound down, which the
// rule does not follow: with 64 ranks 64 rows of 4 adapters 16 against 23 and of
// 64 33 against 36, 128 rows of 8 26 against 25, 256 rows of 8 44 against 29 and
// of one 29 against 22; with 128 ranks 64 rows of 4 23 against 25, 256 of 8 76
// against 36.
AdPlan adapter_plan(int M, int G)
{
    AdPlan p;
    p.few = M <= 256;
    p.sorted = !p.few && G > 1;
    return p;
}

void adapter_shrink(const AdShrinkArgs &a, const AdPlan &plan, int x_dtype, int a_dtype, hipStream_t stream)
{
    with_dtype(x_dtype, [&](auto x) {
        with_dtype(a_dtype, [&](auto w) {
            typedef decltype(x) X;
            typedef decltype(w) A;
            if (plan.few) {
                hipLaunchKernelGGL((ad_shrink_few<X, A>), dim3(a.M, adapter_ranks(a.r) / kAdFewRanks), dim3(kAdFewWaves * 64),
                                   0, stream, a);
                return;
            }
            const unsigned tiles = (unsigned)((a.M + 15LL) / 16);
            const unsigned more = a.order ? (a.G < 256 ? a.G : 256) : 0;      // for adapters that begin inside a tile
            auto launch = [&](auto rt) {
                constexpr int RT = decltype(rt)::value;
                hipLaunchKernelGGL((ad_shrink_tile<X, A, RT>), dim3(tiles + more, (a.r + 16 * RT - 1) / (16 * RT)),
                                   dim3(kAdWaves * 64), 0, stream, a);
            };
            // More ranks a workgroup, which reads x for all of them, if that leaves
            // workgroups enough.  64 ranks of 4096 columns, with 16, 32 and 64 ranks a
            // workgroup: 300 rows 11.3, 12.6 and 16.8 us, 1000 rows 15.8, 13.6 and
            // 16.5, 2011 rows 24.2, 20.7 and 17.8 (fp16 and kept: 18.6 and 21.6 for
            // the latter two), 8192 rows 75, 53 and 46.
            auto enough = [&](int ranks, int least) {
                return a.r > ranks / 2 && (long long)tiles * ((a.r + ranks - 1) / ranks) >= least;
            };
            if (enough(64, 200))
                launch(std::integral_constant<int, 4>{});
            else if (enough(32, 100))
                launch(std::integral_constant<int, 2>{});
            else
                launch(std::integral_constant<int, 1>{});
        });
    });
}

}  // namespace convimg
