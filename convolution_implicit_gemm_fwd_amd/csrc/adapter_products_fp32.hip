// adapter_products_fp32.hip -- adapter_products.hpp for adapters in fp32.
#include "adapter_products.hpp"

namespace convimg {

void gemm_adapters_fp32(const MxGemmArgs &g, const MxAdapterArgs &ad, int out_dtype, hipStream_t stream)
{
    gemm_adapters_of<Fp32>(g, ad, out_dtype, stream);
}

void few_adapters_fp32(const MxFewArgs &g, const MxAdapterArgs &ad, int x_dtype, int out_dtype, hipStream_t stream)
{
    few_adapters_of<Fp32>(g, ad, x_dtype, out_dtype, stream);
}

}  // namespace convimg
