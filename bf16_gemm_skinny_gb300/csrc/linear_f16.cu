// linear_f16.cu -- the FP16 instances of the feed-forward layer products
// (kernels in linear_tcgen05.cuh).
#include "linear_tcgen05.cuh"

namespace bsk {

int launch_linear_f16(const LinearLaunch& g, cudaStream_t stream, char* msg, size_t msg_len)
{
    return launch_linear_type<kTypeF16>(g, stream, msg, msg_len);
}

}  // namespace bsk
