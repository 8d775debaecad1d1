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

// Part of block c: slot 2 c + 1 where the item begins (c == first), else 2 c.
__device__ __forceinline__ long long part_of(int c, int first) { return 2LL * c + (c == first ? 1 : 0); }

__device__ __forceinline__ long long out_row(const AttnParams &p, int row, int t0, int h)
{
    const int tok = p.by_group(row);
    return static_cast<long long>(t0 + tok) * p.q_heads + h * p.group + row - tok * p.group;
}

// Parts of the decode kernel, [16 rows][D].  Block (c, y): row y of the item whose last
// part is in block c of the attention kernel (meta[c]).  A long axis leaves tens of
// parts: the four warps take every fourth one each and meet in shared memory.
template <int D, bool BF16>
__global__ void __launch_bounds__(128)
join_decode_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int kVec = D / 32;
    __shared__ float so[4][D];
    __shared__ float2 sml[4];
    if (threadIdx.x == 0)
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int last = blockIdx.x, row = blockIdx.y;
    const int4 mt = p.meta[2 * last];
    if (mt.x < 0 || row >= mt.y)
        return;
    const int h = p.meta[2 * last + 1].x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, first = mt.x;
    float m = -INFINITY, l = 0.f, o[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e)
        o[e] = 0.f;
    // eight parts at a time: their loads are under way together
    for (int c0 = first + warp; c0 <= last; c0 += 32) {
        float2 ml[8];
        float v[8][kVec];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int c = c0 + 4 * u;
            ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                v[u][e] = 0.f;
            if (c <= last) {
                const long long at = part_of(c, first) * kDecodeRows + row;
                ml[u] = *reinterpret_cast<const float2 *>(p.part_ml + 2 * at);
                const float *src = p.part_o + at * D + lane * kVec;
                if constexpr (kVec == 4) {
                    const float4 q = *reinterpret_cast<const float4 *>(src);
                    v[u][0] = q.x; v[u][1] = q.y; v[u][2] = q.z; v[u][3] = q.w;
                } else {
                    const float2 q = *reinterpret_cast<const float2 *>(src);
                    v[u][0] = q.x; v[u][1] = q.y;
                }
            }
        }
        float mn = m;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            mn = fmaxf(mn, ml[u].x);
        const float base = mn == -INFINITY ? 0.f : mn, a = ex2(m - base);
        m = mn;
        l *= a;
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            o[e] *= a;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const float w = ex2(ml[u].x - base);
            l = fmaf(w, ml[u].y, l);
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                o[e] = fmaf(w, v[u][e], o[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e)
        so[warp][lane * kVec + e] = o[e];
    if (lane == 0)
        sml[warp] = make_float2(m, l);
    __syncthreads();
    if (threadIdx.x * 2 < D) {
        float mm = -INFINITY, ll = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w)
            mm = fmaxf(mm, sml[w].x);
        const float base = mm == -INFINITY ? 0.f : mm;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float a = ex2(sml[w].x - base);
            ll = fmaf(a, sml[w].y, ll);
            o0 = fmaf(a, so[w][2 * threadIdx.x], o0);
            o1 = fmaf(a, so[w][2 * threadIdx.x + 1], o1);
        }
        const long long at = out_row(p, mt.z + row, mt.w, h);
        const float inv = row_inverse(ll);
        reinterpret_cast<uint32_t *>(p.out + at * D)[threadIdx.x] = pack16<BF16>(o0 * inv, o1 * inv);
        if (p.lse && threadIdx.x == 0)
            p.lse[at] = row_log_sum<BF16>(mm, ll);
    }
}

// Parts of the chunk kernel, [D / 4][256 rows][4].  Block (c, y): rows 32 y .. 32 y + 31
// of the item, one per lane; warp w takes values D / 8 w .. D / 8 (w + 1) of them.
template <int D, bool BF16>
__global__ void __launch_bounds__(256)
join_chunk_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int kQuads = D / 32;      // groups of four values per thread
    if (threadIdx.x == 0)
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int last = blockIdx.x;
    const int4 mt = p.meta[2 * last];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = 32 * blockIdx.y + lane;
    if (mt.x < 0 || row >= mt.y)
        return;
    const int h = p.meta[2 * last + 1].x, first = mt.x;
    float m = -INFINITY, l = 0.f;
    float4 o[kQuads];
#pragma unroll
    for (int e = 0; e < kQuads; ++e)
        o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = first; c0 <= last; c0 += 2) {   // two parts at a time
        float2 ml[2];
        float4 v[2][kQuads];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int e = 0; e < kQuads; ++e)
                v[u][e] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c0 + u <= last) {
                const long long at = part_of(c0 + u, first);
                ml[u] = *reinterpret_cast<const float2 *>(p.part_ml + 2 * (at * kChunkRows + row));
#pragma unroll
                for (int e = 0; e < kQuads; ++e)
                    v[u][e] = *reinterpret_cast<const float4 *>(p.part_o + at * (kChunkRows * D) +
                                                                ((warp * kQuads + e) * kChunkRows + row) * 4);
            }
        }
        const float mn = fmaxf(m, fmaxf(ml[0].x, ml[1].x)), base = mn == -INFINITY ? 0.f : mn;
        const float a = ex2(m - base), w0 = ex2(ml[0].x - base), w1 = ex2(ml[1].x - base);
        m = mn;
        l = a * l + (w0 * ml[0].y + w1 * ml[1].y);
#pragma unroll
        for (int e = 0; e < kQuads; ++e) {
            o[e].x = a * o[e].x + (w0 * v[0][e].x + w1 * v[1][e].x);
            o[e].y = a * o[e].y + (w0 * v[0][e].y + w1 * v[1][e].y);
            o[e].z = a * o[e].z + (w0 * v[0][e].z + w1 * v[1][e].z);
            o[e].w = a * o[e].w + (w0 * v[0][e].w + w1 * v[1][e].w);
        }
    }
    const long long at = out_row(p, mt.z + row, mt.w, h);
    const float inv = row_inverse(l);
    uint2 *dst = reinterpret_cast<uint2 *>(p.out + at * D + warp * (D / 8));
#pragma unroll
    for (int e = 0; e < kQuads; ++e)
        dst[e] = make_uint2(pack16<BF16>(o[e].x * inv, o[e].y * inv), pack16<BF16>(o[e].z * inv, o[e].w * inv));
    if (p.lse && warp == 0)
        p.lse[at] = row_log_sum<BF16>(m, l);
}

template <int D, bool BF16>
cudaError_t launch_join(const AttnParams &p, int grid, bool few, int max_rows, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = few ? dim3(grid, max_rows) : dim3(grid, (max_rows + 31) / 32);
    cfg.blockDim = dim3(few ? 128 : 256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return few ? cudaLaunchKernelEx(&cfg, join_decode_kernel<D, BF16>, p)
               : cudaLaunchKernelEx(&cfg, join_chunk_kernel<D, BF16>, p);
}

cudaError_t launch_attn_join(const AttnParams &p, int grid, bool few, int max_rows, cudaStream_t stream)
{
    const bool bf16 = p.kv.dtype == QMM_BF16;
    if (p.kv.head_dim == 128)
        return bf16 ? launch_join<128, true>(p, grid, few, max_rows, stream)
                    : launch_join<128, false>(p, grid, few, max_rows, stream);
    return bf16 ? launch_join<64, true>(p, grid, few, max_rows, stream)
                : launch_join<64, false>(p, grid, few, max_rows, stream);
}

// The decode kernel holds 16 query rows per key head.
bool few_rows(int max_q, int group) { return static_cast<long long>(max_q) * group <= kDecodeRows; }

int attn_grid(bool few, int num_sms) { return few ? kDecodeBlocksPerSm * num_sms : num_sms; }

size_t scratch_bytes(bool few, int head_dim, int num_sms)
{
    const size_t g = attn_grid(few, num_sms), rows = few ? kDecodeRows : kChunkRows;
    return g * 32 + 2 * g * rows * (head_dim + 2) * 4;
}

// Work a block takes at least, in units: below this a split costs more (a second
// kernel, the partial results) than the longer walk.  Decode kernel (blocks of four warps): one
// token over 30000 keys of one key head 12.5 us, with 2 units 16.1, 8 13.2, 12 15.4; over 16000
// of four 12.9, with 2 12.0, 8 13.5, 12 16.6.  Chunk kernel, 30 items of up to 12 units: 18.1 us,
// with 6 20.4.
constexpr int kMinDecodeUnits = 5, kMinChunkUnits = 4;

// Work of the longest item (setup and units) up to which blocks of the chunk kernel take
// whole items: no joining kernel, against blocks of unequal work by up to one item.  Four
// sequences of up to 1000 tokens, work 10: 47.8 us, split 49.5; seven chunks with a
// window of 1000, work 12: 35.6, split 36.8; prompts of 2048, work 18: 49.9, split 41.6.
constexpr int kUnsplitWork = 12;

// The same where every item has a block of its own (20 items of up to 6 units: 14.6 us,
// split 19.3).
constexpr int kWholeWork = 10;

// Whole items in clusters against a split over all blocks: a cluster's block walks
// units / c, a split one units * items / blocks and the joining kernel's time, some 5
// units; and not more than 12 units, since whole items are not balanced where lengths
// differ.  One token over 8000 keys 11.6 us in clusters (8 units), 12.0 split; 16000 keys
// (16) 18.9 and 14.6; eight over 3000 (12) 15.8 and 18.4.
constexpr int kJoinUnits = 5, kMostUnits = 12;

// What starting an item costs a block, in units, and the items (in 16 keys at head size
// 128) that are short enough for one block however many they are.  Blocks of one warp take
// four times the units of those of four and fit seven to an SM instead of two: 1728 items
// of 4 keys 8.0 us against 20.5, 2048 of 256 keys 44 against 51, 512 of 256 keys 16.4
// against 13.2.
constexpr int kStartUnits = 3, kWholeKeys = 16;

// Blocks per item of the decode kernel, and their warps, where every item gets a cluster
// (or block) of its own: clusters of the largest size that all run at once (eight
// clusters of eight on 64 SMs do, sixteen on 128 do not: 12.0 us for 24 rows over 1000
// keys, 7.9 in sixteen of four).  Eight warps a block where an SM is free for each: one
// token over 2000 keys 6.2 us against 7.4 with four, over 4000 8.1 against 10.4.  Items
// short enough for one block go there however many they are, to blocks of four warps or of
// one.  0: the axis is split over all blocks.  A window bounds the items' keys (16 tokens,
// the last 500 of 4000 keys: 8.1 us, 11.9 without).
int decode_cluster(const AttnParams &p, long long items, long long max_kv, int num_sms, int *warps)
{
    const bool bf16 = p.kv.dtype == QMM_BF16;
    // an item's keys at most, and one unit more where a window may start inside one
    const long long span = p.window > 0 ? std::min(max_kv, static_cast<long long>(p.window) + kDecodeRows / p.group + 1) : max_kv;
    const int more = span < max_kv;
    for (*warps = 8; *warps >= 4; *warps /= 2) {
        const int keys = decode_keys(p.kv.head_dim, *warps);
        const long long units = (span + keys - 1) / keys + more, blocks = *warps == 8 ? num_sms : kDecodeBlocksPerSm * num_sms;
        for (int c = kMaxCluster; c >= 1; c /= 2)
            if (items * c <= blocks && (c == 1 || c / 2 < units) && (units + c - 1) / c <= kMostUnits &&
                (units + c - 1) / c <= items * units / blocks + kJoinUnits &&
                (c == 1 || items <= attn_decode_clusters(p.kv.head_dim, bf16, *warps, c)))
                return c;
    }
    // longer: the axis is split over two blocks of four warps per SM, which the split's grid is
    // sized for (128 sequences of 300 to 4096 keys, 8 key heads: 175 us; on as many blocks of
    // one warp, a quarter of the copies in flight, 373)
    *warps = 4;
    if (span > kWholeKeys * decode_keys(p.kv.head_dim, 1) || items > 0x7fffffff)
        return 0;
    // more short items than blocks at once: each costs its block a start and its units
    const auto rounds = [&](int w, int blocks_per_sm) {
        const int keys = decode_keys(p.kv.head_dim, w);
        const long long blocks = static_cast<long long>(blocks_per_sm) * num_sms;
        return (items + blocks - 1) / blocks * (kStartUnits + (span + keys - 1) / keys + more);
    };
    if (rounds(1, kNarrowBlocksPerSm) < rounds(4, kDecodeBlocksPerSm))
        *warps = 1;
    return 1;
}

}  // namespace

size_t attn_workspace_bytes(int q_heads, int kv_heads, int head_dim, int max_q, int num_sms)
{
    return scratch_bytes(few_rows(std::max(1, max_q), q_heads / kv_heads), head_dim, num_sms);
}

cudaError_t attn_dispatch(AttnParams &p, int max_q, long long max_kv, void *workspace, int num_sms, cudaStream_t stream)
{
    // no sequence has more tokens than the batch: a caller's large bound adds no row tiles, and
    // the rows of a sequence are counted in 32 bits (qmm_paged_attn checks tokens * group)
    max_q = std::max(1, std::min(max_q, p.kv.tokens));
    const long long most = static_cast<long long>(p.kv.blocks) * p.kv.page_size, q_rows = static_cast<long long>(max_q) * p.group;
    if (max_kv <= 0 || max_kv > most)
        max_kv = most;
    if (p.window >= most)   // no position lies further back
        p.window = 0;
    // the decode kernel's items
    const long long dtiles = (q_rows + kDecodeRows - 1) / kDecodeRows, ditems = p.kv.batch * dtiles * p.kv.kv_heads;
    int warps;
    const int cluster = decode_cluster(p, ditems, max_kv, num_sms, &warps);
    // more rows go to it too where its items, sixteen rows each, all run at once: it
    // starts faster and needs no join (64 tokens over 1000 keys 11.4 us against the chunk
    // kernel's 18.3, 128 over 128 6.0 against 8.0; but 4 x 50 over 200, 416 items on 304
    // blocks, 13.9 against 9.6, and 5 over 4000 of 32 sequences, split, 243 against 94)
    // (and queries that the chunk kernel's tensor copies do not take: groups of over 128
    // heads, strides of zero)
    const bool few = few_rows(max_q, p.group) || (cluster > 0 && ditems * cluster <= kDecodeBlocksPerSm * num_sms) ||
                     !attn_set_q_tma(p);
    const int rows = few ? kDecodeRows : 2 * chunk_stream_rows(p.group), keys = few ? decode_keys(p.kv.head_dim, warps) : kChunkKeys;
    const int setup = few ? kDecodeSetup : kChunkSetup;
    p.tile_rows = rows;
    p.row_tiles = static_cast<int>((q_rows + rows - 1) / rows);
    p.by_group = fast_div(p.group);
    p.by_tiles = fast_div(p.row_tiles);
    p.by_page = fast_div(p.kv.page_size);
    p.warps = warps;
    p.same_page = p.kv.page_size % (decode_keys(p.kv.head_dim, 4) / 4) == 0;
    p.min_chunk = few ? kMinDecodeUnits : kMinChunkUnits;
    const long long items = static_cast<long long>(p.kv.batch) * p.row_tiles * p.kv.kv_heads;
    long long longest = (max_kv + keys - 1) / keys;
    if (p.window > 0)   // the keys that a tile's tokens see between them
        longest = std::min(longest, (static_cast<long long>(p.window) + rows / p.group + 1) / keys + 2);
    // one block or cluster per item where no item is long enough to be split over more
    p.cluster = few && cluster > 0 ? cluster : 1;
    int grid = attn_grid(few, num_sms);
    p.whole = few ? cluster > 0 : items <= grid ? longest + setup <= kWholeWork : longest + setup <= kUnsplitWork;
    p.unsplit = !few && p.whole && items > grid;
    if (p.whole && !p.unsplit)
        grid = static_cast<int>(items) * p.cluster;
    else if (p.unsplit)
        p.min_chunk = 1;
    else if (items * (longest + setup) < static_cast<long long>(grid) * p.min_chunk)
        grid = static_cast<int>((items * (longest + setup) + p.min_chunk - 1) / p.min_chunk);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const size_t g = attn_grid(few, num_sms);
    p.meta = reinterpret_cast<int4 *>(ws);
    p.part_ml = reinterpret_cast<float *>(ws + g * 32);
    p.part_o = p.part_ml + 2 * g * (few ? kDecodeRows : kChunkRows) * 2;
    if (!few)
        attn_set_tma(p);
    cudaError_t e = few ? launch_attn_decode(p, grid, stream) : launch_attn_chunk(p, grid, stream);
    if (e != cudaSuccess || p.whole)
        return e;
    return launch_attn_join(p, grid, few, static_cast<int>(std::min(static_cast<long long>(rows), q_rows)), stream);
}

}  // namespace qmm
