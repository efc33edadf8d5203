// adapter_products.hpp -- the linear layer's products with the adapters' second
// half inside, for one type of the adapters (a translation unit each).
#pragma once

#include "adapter.hpp"

namespace convimg {

template <typename T>
MxAdapters<T> adapters_of(const MxAdapterArgs &a)
{
    MxAdapters<T> t;
    static_cast<MxAdapterArgs &>(t) = a;
    return t;
}

template <typename T>
void gemm_adapters_of(MxGemmArgs g, const MxAdapterArgs &ad, int out_dtype, hipStream_t stream)
{
    with_dtype(out_dtype, [&](auto o) {
        with_shape(shape_of(tiles_of(g.M, g.N), g.kb), [&](auto shape) {
            typedef decltype(shape) S;
            const unsigned grid = gemm_grid(g, S::BM, S::BN);
            hipLaunchKernelGGL((mx_gemm_tile_adapters<S, decltype(o), T>), dim3(grid), dim3(S::threads), 0, stream, g,
                               adapters_of<T>(ad));
        });
    });
}

template <typename T>
void few_adapters_of(const MxFewArgs &g, const MxAdapterArgs &ad, int x_dtype, int out_dtype, hipStream_t stream)
{
    const int pairs = (g.kb + 7) / 8, waves = pairs < kMxFewWaves ? pairs : kMxFewWaves;
    with_dtype(x_dtype, [&](auto x) {
        with_dtype(out_dtype, [&](auto o) {
            hipLaunchKernelGGL((mx_gemm_few<decltype(x), decltype(o), MxAdapters<T>>), dim3((g.N + 15) / 16),
                               dim3(waves * 64), 0, stream, g, adapters_of<T>(ad));
        });
    });
}

}  // namespace convimg
