// adapter_products_bf16.hip -- adapter_products.hpp for adapters in bf16.
#include "adapter_products.hpp"

namespace convimg {

void gemm_adapters_bf16(const MxGemmArgs &g, const MxAdapterArgs &ad, int out_dtype, hipStream_t stream)
{
    gemm_adapters_of<Bf16>(g, ad, out_dtype, stream);
}

void few_adapters_bf16(const MxFewArgs &g, const MxAdapterArgs &ad, int x_dtype, int out_dtype, hipStream_t stream)
{
    few_adapters_of<Bf16>(g, ad, x_dtype, out_dtype, stream);
}

}  // namespace convimg
