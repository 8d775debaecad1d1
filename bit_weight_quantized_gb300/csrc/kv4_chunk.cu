// kv4_chunk.cu -- the kernel for many query rows over the 4-bit paged cache: six warps copy codes
// and turn them into the tiles that tensor copies bring from a 16-bit cache.
#include "attn_chunk.cuh"

namespace qmm {

cudaError_t launch_kv4_chunk(const Kv4AttnParams &p, int grid, cudaStream_t stream)
{
    return launch_chunk_form<true>(p, grid, stream);
}

}  // namespace qmm
