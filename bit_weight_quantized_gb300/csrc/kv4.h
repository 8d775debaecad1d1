// kv4.h -- host interface of the 4-bit paged key / value cache kernels
// (qmm_kv4_append, qmm_kv4_read, qmm_kv4_attn).
#pragma once

#include "paged.h"

namespace qmm {

// Values that share a scale and a zero.
constexpr int kKv4Group = 64;

// The scales of a 4-bit cache: element (page, slot, head) at page * page_stride + ...; a
// key's scales, then its value's, one per group.  (The codes are qmm_paged_kv's k and v, with
// strides in bytes.)
struct Kv4Scales {
    uint16_t *base;
    long long page, slot, head;
};

struct Kv4AppendParams : AppendParams {
    Kv4Scales sc;
    const uint16_t *q_norm, *k_norm;   // weights of the norms, or nullptr
    float eps, one;                    // one: 1
};

struct Kv4ReadParams {
    qmm_paged_kv kv;
    Kv4Scales sc;
    uint16_t *k, *v;                   // dense [tokens][kv_heads][D]
    int *status;
    int rows;                          // tokens per block
    int wide;                          // outputs take 32-byte stores
    // all visible keys (kv4_unpack): room per sequence and head, window, the block table to write
    int32_t *table;
    int cap, window;
    FastDiv by_page, by_heads;
};

struct Kv4AttnParams : AttnParams {
    Kv4Scales sc;
    // places of codes in 32 bits (kernel for few rows): the strides in units of `unit` bytes, the
    // largest power of two that divides them
    uint32_t unit, page_units, slot_units;
};

cudaError_t launch_kv4_append(const Kv4AppendParams &p, cudaStream_t stream);
// The batch's tokens, or with p.table all keys that they see, laid out for attn_chunk.cuh.
cudaError_t launch_kv4_read(Kv4ReadParams &p, int num_sms, cudaStream_t stream);

// Keys per unit of the kernel for few rows: a warp's stage holds 4 KB of codes.
__host__ __device__ constexpr int kv4_keys(int head_dim, int warps) { return 4096 / head_dim * warps; }
// Blocks of it per SM, of four or eight warps (8 rows take 128 registers a thread, 16 all 255).
__host__ __device__ constexpr int kv4_blocks_per_sm(int rows, int warps) { return (rows == 8 ? 16 : 8) / warps; }

// Clusters of `cluster` blocks of eight warps that run at once on the current device.
int kv4_decode_clusters(int head_dim, bool bf16, int rows, int cluster);

// p.warps: 4 or 8; p.tile_rows: 8 or 16.
cudaError_t launch_kv4_decode(const Kv4AttnParams &p, int grid, cudaStream_t stream);

cudaError_t launch_kv4_chunk(const Kv4AttnParams &p, int grid, cudaStream_t stream);

// Sets the units; false where places do not fit.
bool kv4_set_units(Kv4AttnParams &p);
size_t kv4_attn_workspace_bytes(int q_heads, int kv_heads, int head_dim, int max_q, int num_sms);
// What a call of these sizes takes beyond that to convert its keys once; 0 where it would not.
size_t kv4_attn_unpack_bytes(int batch, int tokens, int group, int kv_heads, int head_dim, int max_q, long long max_kv,
                             int sinks);
// workspace: as many bytes as kv4_attn_workspace_bytes() says, and `more`.
cudaError_t kv4_attn_dispatch(Kv4AttnParams &p, int max_q, long long max_kv, void *workspace, size_t more, int num_sms,
                              cudaStream_t stream);

}  // namespace qmm
