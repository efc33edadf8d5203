// adapter.hpp -- the passes of low-rank adapters that are launches of their
// own: h = down x with the quantisation of x, and the adapters' gradients.
#pragma once

#include "mxfp4_plan.hpp"

namespace convimg {

struct AdShrinkArgs {
    const void *x;                      // dense rows ldx apart
    const void *down;                   // [G][r][K]
    const float *scale;                 // [G]
    const int *key;                     // [M]: the adapter at each place of h and codes
    const int *order, *start;           // adapter_sort: [M], the row at each place; NULL for their own order
    float *h;                           // [M][adapter_ranks(r)]
    unsigned char *terms;               // h for the products (MxAdapterArgs), or NULL
    float *kept;                        // [M][r]: h in the rows' own order, too, or NULL
    unsigned char *codes, *scales;      // MXFP4 rows of x to write, or NULL
    unsigned char *codes8, *scales8;    // MXINT8 rows of x to write, in their own order, or NULL
    long long ldx;
    int M, K, G, r;
};

// How the rows of a call are walked: a row a workgroup, in their own order, or
// 16 at a time, then sorted by adapter if there are several.
struct AdPlan {
    bool few, sorted;
};
AdPlan adapter_plan(int M, int G);
void adapter_shrink(const AdShrinkArgs &a, const AdPlan &plan, int x_dtype, int a_dtype, hipStream_t stream);

// The rows sorted by adapter, those without one last, rows of one adapter by
// their numbers: order [M] (and as much again behind it), key [M], the adapter
// at each place or -1, and start [G + 1], the first place of each adapter and of
// the rows without.  With `nan` a 0 there.
void adapter_sort(const int *ids, int M, int G, int *order, int *key, int *start, int *nan, hipStream_t stream);

// One operand of the gradients: out[g][i][c] = scale_g * sum over the rows m
// of g of u[m][i] * v[m][c].
struct AdGradArgs {
    const float *u;                     // [M] rows of r
    const void *v;                      // dense rows ldv apart, or MXINT8 codes
    const unsigned char *vs;            // their scale bytes
    const int *order, *key, *start;     // adapter_sort
    const float *scale;
    float *out;                         // [G][r][C]
    float *part;                        // [chunks][2][r][C]
    int *nan;                           // set if a sum is NaN; 0 before
    long long ldv;
    int M, C, G, r;
    int u_sorted, u_ld;                 // u's rows are in sorted order; their stride
    int per, chunks;                    // sorted rows a chunk
    int tiles, ranks;                   // of 128 columns, of the ranks that a workgroup takes
};

}  // namespace convimg
