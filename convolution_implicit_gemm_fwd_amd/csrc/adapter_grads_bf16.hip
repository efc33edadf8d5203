// adapter_grads_bf16.hip -- adapter_grads.hpp for dy in bf16.
#include "adapter_grads.hpp"

namespace convimg {

void adapter_grads_bf16(const AdGradArgs &up, const AdGradArgs &down, int x_dtype, hipStream_t stream)
{
    adapter_grads_of<Bf16>(up, down, x_dtype, stream);
}

}  // namespace convimg
