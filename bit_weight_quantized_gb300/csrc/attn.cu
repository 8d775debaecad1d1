// attn.cu -- qmm_paged_attn: kernel choice, split sizes, and the kernel that joins
// the partial results of items split over several blocks.
//
// Joining is the softmax's own sum: with each part's maximum m_c, sum l_c and
// unnormalized output o_c (both relative to 2^m_c),
//   m = max m_c,  w_c = 2^(m_c - m),  out = sum w_c o_c / sum w_c l_c,
// in fp32, parts in the order of the keys.
#include <algorithm>

#include "paged.cuh"

namespace qmm {

namespace {

constexpr int kCombineWarps = 4;

// Block (c, y): the item whose last part is in block c of the attention kernel
// (meta[c]); one warp per row.
template <int D, int ROWS, int KEYS, bool BF16>
__global__ void __launch_bounds__(32 * kCombineWarps)
attn_combine_kernel(const __grid_constant__ AttnParams p)
{
    constexpr float kShift = BF16 ? 0.f : 7.f;
    constexpr int kVec = D / 32;
    if (threadIdx.x == 0)
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int last = blockIdx.x;
    const int4 mt = p.meta[last];
    if (mt.x < 0)
        return;
    const int lane = threadIdx.x & 31, first = mt.z;
    const RowTile r = row_tile<ROWS, KEYS>(p, mt.x);
    for (int row = blockIdx.y * kCombineWarps + (threadIdx.x >> 5); row < r.rows; row += gridDim.y * kCombineWarps) {
        // part of block c: slot 2 c + 1 where the item begins (c == first), else 2 c
        auto part = [&](int c) { return (2LL * c + (c == first ? 1 : 0)) * ROWS + row; };
        float m = -INFINITY;
        for (int c = first + lane; c <= last; c += 32)
            m = fmaxf(m, p.part_ml[2 * part(c)]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float base = m == -INFINITY ? 0.f : m;
        float l = 0.f, o[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            o[e] = 0.f;
#pragma unroll 4
        for (int c = first; c <= last; ++c) {
            const float2 ml = *reinterpret_cast<const float2 *>(p.part_ml + 2 * part(c));
            const float *src = p.part_o + part(c) * D + lane * kVec;
            float v[kVec];
            if constexpr (kVec == 4) {
                const float4 q = *reinterpret_cast<const float4 *>(src);
                v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
            } else {
                const float2 q = *reinterpret_cast<const float2 *>(src);
                v[0] = q.x; v[1] = q.y;
            }
            const float w = ex2(ml.x - base);
            l = fmaf(w, ml.y, l);
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                o[e] = fmaf(w, v[e], o[e]);
        }
        const int rr = r.row0 + row, tok = rr / p.group;
        const long long at = static_cast<long long>(r.t0 + tok) * p.q_heads + mt.y * p.group + rr - tok * p.group;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        uint32_t w[kVec / 2];
#pragma unroll
        for (int e = 0; e < kVec / 2; ++e)
            w[e] = pack16<BF16>(o[2 * e] * inv, o[2 * e + 1] * inv);
        uint16_t *dst = p.out + at * D + lane * kVec;
        if constexpr (kVec == 4)
            *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint32_t *>(dst) = w[0];
        if (p.lse && lane == 0)
            p.lse[at] = l > 0.f ? (m - kShift + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
}

template <int D, int ROWS, int KEYS, bool BF16>
cudaError_t launch_combine(const AttnParams &p, int grid, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    const int tile_rows = std::min(ROWS, p.row_tiles * ROWS);
    cfg.gridDim = dim3(grid, (tile_rows + 4 * kCombineWarps - 1) / (4 * kCombineWarps) * (ROWS > 16 ? 1 : 4));
    cfg.blockDim = dim3(32 * kCombineWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_combine_kernel<D, ROWS, KEYS, BF16>, p);
}

template <int ROWS, int KEYS>
cudaError_t launch_combine_rows(const AttnParams &p, int grid, cudaStream_t stream)
{
    const bool bf16 = p.kv.dtype == QMM_BF16;
    if (p.kv.head_dim == 128)
        return bf16 ? launch_combine<128, ROWS, KEYS, true>(p, grid, stream)
                    : launch_combine<128, ROWS, KEYS, false>(p, grid, stream);
    return bf16 ? launch_combine<64, ROWS, KEYS, true>(p, grid, stream)
                : launch_combine<64, ROWS, KEYS, false>(p, grid, stream);
}

// The decode kernel holds 16 query rows per key head.
bool few_rows(int max_q, int group) { return static_cast<long long>(max_q) * group <= kDecodeRows; }

int attn_grid(bool few, int num_sms) { return few ? kDecodeBlocksPerSm * num_sms : num_sms; }

size_t scratch_bytes(bool few, int head_dim, int num_sms)
{
    const size_t g = attn_grid(few, num_sms), rows = few ? kDecodeRows : kChunkRows;
    return g * 16 + 2 * g * rows * (head_dim + 2) * 4;
}

// Work a block takes at least, in units: below this a split costs more (a second kernel,
// the partial results) than the longer walk.
constexpr int kMinDecodeUnits = 5, kMinChunkUnits = 4;

}  // namespace

cudaError_t launch_attn_combine(const AttnParams &p, int grid, int rows, cudaStream_t stream)
{
    return rows == kDecodeRows ? launch_combine_rows<kDecodeRows, kDecodeKeys>(p, grid, stream)
                               : launch_combine_rows<kChunkRows, kChunkKeys>(p, grid, stream);
}

size_t attn_workspace_bytes(int q_heads, int kv_heads, int head_dim, int max_q, int num_sms)
{
    return scratch_bytes(few_rows(max_q, q_heads / kv_heads), head_dim, num_sms);
}

cudaError_t attn_dispatch(AttnParams &p, int max_q, long long max_kv, void *workspace, int num_sms, cudaStream_t stream)
{
    const bool few = few_rows(max_q, p.group);
    const int rows = few ? kDecodeRows : kChunkRows, keys = few ? kDecodeKeys : kChunkKeys;
    const int setup = few ? kDecodeSetup : kChunkSetup;
    p.row_tiles = static_cast<int>((static_cast<long long>(max_q) * p.group + rows - 1) / rows);
    p.min_chunk = few ? kMinDecodeUnits : kMinChunkUnits;
    const long long items = static_cast<long long>(p.kv.batch) * p.row_tiles * p.kv.kv_heads;
    const long long most = static_cast<long long>(p.kv.blocks) * p.kv.page_size;
    if (max_kv <= 0 || max_kv > most)
        max_kv = most;
    const long long longest = (max_kv + keys - 1) / keys;      // units of the longest item
    // one block per item where no item is long enough to be split
    p.whole = longest + setup <= p.min_chunk && items <= 0x7fffffff;
    int grid = attn_grid(few, num_sms);
    if (p.whole)
        grid = static_cast<int>(items);
    else if (items * (longest + setup) < static_cast<long long>(grid) * p.min_chunk)
        grid = static_cast<int>((items * (longest + setup) + p.min_chunk - 1) / p.min_chunk);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const size_t g = attn_grid(few, num_sms);
    p.meta = reinterpret_cast<int4 *>(ws);
    p.part_ml = reinterpret_cast<float *>(ws + g * 16);
    p.part_o = p.part_ml + 2 * g * rows * 2;
    cudaError_t e = few ? launch_attn_decode(p, grid, stream) : launch_attn_chunk(p, grid, stream);
    if (e != cudaSuccess || p.whole)
        return e;
    return launch_attn_combine(p, grid, rows, stream);
}

}  // namespace qmm
