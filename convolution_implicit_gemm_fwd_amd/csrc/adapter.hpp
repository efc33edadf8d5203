// adapter.hpp -- the passes of low-rank adapters that are launches of their
// own: h = down x with the quantisation of x, and the adapters' gradients.
#pragma once

#include "mxfp4_plan.hpp"

namespace convimg {

struct AdShrinkArgs {
    const void *x;                      // dense rows ldx apart
    const void *down;                   // [G][r][K]
    const int *ids;                     // [M]
    float *h;                           // [splits][M][r]
    unsigned char *codes, *scales;      // MXFP4 rows of x to write, or NULL
    unsigned char *codes8, *scales8;    // MXINT8 rows of x to write, or NULL
    long long ldx;
    int M, K, G, r;
};

// Parts of the columns whose sums the pass leaves apart.
int adapter_splits(int M, int K, bool whole);
void adapter_shrink(const AdShrinkArgs &a, int x_dtype, int a_dtype, int splits, hipStream_t stream);

// One operand of the gradients: out[g][i][c] = scale_g * sum over the rows m
// with ids[m] = g of u[m][i] * v[m][c].
struct AdGradArgs {
    const float *u;                     // [M][r]
    const void *v;                      // dense rows ldv apart, or MXINT8 codes
    const unsigned char *vs;            // their scale bytes
    const int *ids;
    const float *scale;
    float *out;                         // [G][r][C]
    float *part;                        // [splits][G][r][C]
    int *count;                         // [splits][G]: rows of the adapter in the part
    long long ldv;
    int M, C, G, r;
};

int adapter_grad_splits(int M, int C, int G, int r);
void adapter_grad(const AdGradArgs &a, int v_dtype, int splits, hipStream_t stream);

}  // namespace convimg
