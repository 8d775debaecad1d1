// paged.h -- host interface of the paged key / value cache kernels
// (qmm_kv_append, qmm_paged_attn).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/qmm.h"

namespace qmm {

// Division of 0 <= n < 2^31 by a number known at launch, as a high product and a shift
// (Granlund and Montgomery, "Division by invariant integers using multiplication"): a
// division by a variable is some 30 dependent instructions.  l = ceil(log2 d), mul =
// ceil(2^(31 + l) / d) < 2^32: the product's error, n / 2^(31 + l), is below 1 / d.
struct FastDiv {
    uint32_t mul, shift, one;   // one: d = 1
#ifdef __CUDACC__
    __device__ __forceinline__ int operator()(int n) const
    {
        return one ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), mul) >> shift);
    }
#endif
};

inline FastDiv fast_div(int d)
{
    FastDiv f = {0, 0, d == 1};
    if (d > 1) {
        int l = 1;
        while ((1LL << l) < d)
            ++l;
        f.mul = static_cast<uint32_t>(((1ULL << (31 + l)) + static_cast<uint64_t>(d) - 1) / static_cast<uint64_t>(d));
        f.shift = static_cast<uint32_t>(l - 1);
    }
    return f;
}

struct AppendParams {
    qmm_paged_kv kv;
    const uint16_t *k, *v, *q;
    uint16_t *q_out;
    const float *cos_sin;          // fp32 [rope_len][rot]: cosines, then sines
    int *status;
    long long k_stride, v_stride, q_stride;
    int q_heads, rot, rope_len, interleaved;
    FastDiv by_page;
};

cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t stream);

struct AttnParams {
    // the cache as [page and head][slot / 8][d / 64][slot % 8][d % 64] for tensor copies
    // of `box` slots (chunk kernel; box = 0: no tensor copies); page i, head h is
    // index i * page_step + h
    alignas(64) CUtensorMap tmk, tmv;
    alignas(64) CUtensorMap tmq;   // the queries as [token][head][D], boxes of one stream's rows (chunk kernel)
    int box, page_step;
    qmm_paged_kv kv;
    const uint16_t *q;
    uint16_t *out;
    float *lse;                    // or nullptr
    int *status;
    float *part_o;                 // [2 grid] partial outputs of a row tile (unnormalized)
    float *part_ml;                // [2 grid][rows per tile][2] their maximum and sum
    int4 *meta;                    // [grid][2] the item whose last part block c holds
    long long q_stride;
    float scale_log2;              // scale * log2(e): the softmax works in powers of two
    int q_heads, group;            // query heads, query heads per key head
    int causal, window;
    int sinks;                     // first tokens that a window leaves visible (4-bit cache)
    int tile_rows;                 // rows per tile
    int row_tiles;                 // row tiles per sequence (of the longest one)
    FastDiv by_group, by_tiles, by_page;   // divisions by group, row_tiles, page_size
    int whole;                     // every item in one cluster or block: no partial results
    int unsplit;                   // whole items, several per block (chunk kernel)
    int cluster;                   // blocks per cluster (decode kernel, whole items)
    int warps;                     // of a block of the decode kernel: 1, 4 or 8
    int same_page;                 // every warp tile of the decode kernel lies in one page
    int min_chunk;                 // work a block takes at least, in units
};

// Sizes of one kernel's work items: query rows per tile, keys per unit.
constexpr int kDecodeRows = 16;
// (decode kernel: 8 KB of K and V per warp)
__host__ __device__ constexpr int decode_keys(int head_dim, int warps) { return (head_dim == 64 ? 32 : 16) * warps; }
constexpr int kChunkRows = 256, kChunkKeys = 128;
// (chunk kernel: whole tokens' rows, at most 128 in each of its two streams)
__host__ __device__ constexpr int chunk_stream_rows(int group) { return 128 / group * group; }
// What starting and finishing an item costs, in units (see find_share).  Chunk kernel:
// about 5000 cycles against 2400 a unit; a 2048-token prompt takes 45.7, 41.6, 42.5 and
// 42.9 us with 1 to 4, one of 8192 405, 338, 336 and 340.
constexpr int kDecodeSetup = 1, kChunkSetup = 2;

// Blocks per cluster of the decode kernel at most.
constexpr int kMaxCluster = 8;

// Blocks of the decode kernel per SM (what it is sized for), of four warps and of one.
constexpr int kDecodeBlocksPerSm = 2, kNarrowBlocksPerSm = 7;

// Clusters of `cluster` (2, 4, 8) blocks of `warps` warps of the decode kernel that run at
// once on the current device.
int attn_decode_clusters(int head_dim, bool bf16, int warps, int cluster);

cudaError_t launch_attn_decode(const AttnParams &p, int grid, cudaStream_t stream);
cudaError_t launch_attn_chunk(const AttnParams &p, int grid, cudaStream_t stream);
// Joins the partial results of a split call of `grid` blocks; few: parts of the decode kernel.
cudaError_t launch_attn_join(const AttnParams &p, int grid, bool few, int max_rows, cudaStream_t stream);

// Sets p.box and the tensor maps where the cache takes tensor copies.
void attn_set_tma(AttnParams &p);
// Tensor map of the queries (chunk kernel); false where there can be none.
bool attn_set_q_tma(AttnParams &p);

// Scratch of a call, and the whole call: kernel choice, split and launches.
size_t attn_workspace_bytes(int q_heads, int kv_heads, int head_dim, int max_q, int num_sms);
cudaError_t attn_dispatch(AttnParams &p, int max_q, long long max_kv, void *workspace, int num_sms,
                          cudaStream_t stream);

}  // namespace qmm
