// attn_chunk.cu -- the kernel for many query rows over the 16-bit paged cache.
#include "attn_chunk.cuh"

namespace qmm {

cudaError_t launch_attn_chunk(const AttnParams &p, int grid, cudaStream_t stream)
{
    return launch_chunk_form<false>(p, grid, stream);
}

}  // namespace qmm
