// adapter.hpp -- the passes of low-rank adapters that are launches of their
// own: h = down x with the quantisation of x, and the adapters' gradients.
#pragma once

#include "mxfp4_plan.hpp"

namespace convimg {

struct AdShrinkArgs {
    const void *x;                      // dense rows ldx apart
    const void *down;                   // [G][r][K]
    const int *ids;                     // [M]
    const int *order;                   // [M]: the row at each place of h and codes, or NULL for their own order
    float *h;                           // [splits][M][r]
    float *kept;                        // h in the rows' own order, too, or NULL
    unsigned char *codes, *scales;      // MXFP4 rows of x to write, or NULL
    unsigned char *codes8, *scales8;    // MXINT8 rows of x to write, in their own order, or NULL
    long long ldx;
    int M, K, G, r;
};

// How the rows of a call are walked.
struct AdPlan {
    bool few;          // a row a workgroup, in their own order
    bool sorted;       // by adapter
    int splits;        // parts of the columns whose sums h leaves apart
};
AdPlan adapter_plan(int M, int K, int G, bool keep);
void adapter_shrink(const AdShrinkArgs &a, const AdPlan &plan, int x_dtype, int a_dtype, hipStream_t stream);

// The rows sorted by adapter, those without one last, a row's place among those
// of its adapter by its number: order [M] (and as much again behind it), and
// start [G + 1], the first place of each adapter and of the rows without, or NULL.
void adapter_sort(const int *ids, int M, int G, int *order, int *start, hipStream_t stream);

// One operand of the gradients: out[g][i][c] = scale_g * sum over the rows m
// of g of u[m][i] * v[m][c].
struct AdGradArgs {
    const float *u;                     // [M][r]
    const void *v;                      // dense rows ldv apart, or MXINT8 codes
    const unsigned char *vs;            // their scale bytes
    const int *ids, *order, *start;     // adapter_sort
    const float *scale;
    float *out;                         // [G][r][C]
    float *part;                        // [chunks][2][r][C]
    long long ldv;
    int M, C, G, r;
    int u_sorted;                       // u's rows are in sorted order
    int per, chunks;                    // sorted rows a chunk
};

int adapter_grad_per(int M, int C, int r);
void adapter_grad(const AdGradArgs &a, int v_dtype, hipStream_t stream);

}  // namespace convimg
