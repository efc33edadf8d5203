// adapter_grads_fp32.hip -- adapter_grads.hpp for dy in fp32.
#include "adapter_grads.hpp"

namespace convimg {

void adapter_grads_fp32(const AdGradArgs &up, const AdGradArgs &down, int x_dtype, hipStream_t stream)
{
    adapter_grads_of<Fp32>(up, down, x_dtype, stream);
}

}  // namespace convimg
