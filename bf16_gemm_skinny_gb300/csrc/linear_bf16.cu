// linear_bf16.cu -- the BF16 instances of the feed-forward layer products
// (kernels in linear_tcgen05.cuh).
#include "linear_tcgen05.cuh"

namespace bsk {

int launch_linear_bf16(const LinearLaunch& g, cudaStream_t stream, char* msg, size_t msg_len)
{
    return launch_linear_type<kTypeBF16>(g, stream, msg, msg_len);
}

}  // namespace bsk
