// adapter_grads_fp16.hip -- adapter_grads.hpp for dy in fp16.
#include "adapter_grads.hpp"

namespace convimg {

void adapter_grads_fp16(const AdGradArgs &up, const AdGradArgs &down, int x_dtype, hipStream_t stream)
{
    adapter_grads_of<Fp16>(up, down, x_dtype, stream);
}

}  // namespace convimg
