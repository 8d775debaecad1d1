// kv_append.cu -- storing new keys and values in the paged cache, keys (and the
// queries beside them) rotated by their positions on the way.
//
//   a' = a cos - b sin,  b' = b cos + a sin   for the pairs (x[i], x[i + rot/2]) or
//   (x[2i], x[2i + 1]), i < rot/2, in fp32 with one rounding; the rest is copied.
//
// Bound by memory: every value is read once and written once, with 16-byte
// accesses.  A block serves one token.  Its threads form columns of head_dim / 16:
// thread i of a column owns two 8-value chunks of a head, the two halves of eight
// pairs (chunks i and i + rot/16 of the half-split order, chunks 2i and 2i + 1 of
// the interleaved one), so that both orders use cosines and sines 8i .. 8i + 7.
// They are loaded once per thread and serve every head the thread's column walks
// (queries, then keys, then values), kBatch heads at a time.  The token's sequence is
// found by a warp-wide count over cu_q, so a call costs three dependent memory round
// trips (cu_q and kv_len; the page and the rotations; the stores); the first heads are
// loaded before the first of them returns.  One token of 48 heads takes 2.3 us, 64
// tokens 2.7 us in a row.
#include "paged.cuh"

namespace qmm {

namespace {

// Threads per token and heads in flight per thread: 8192 tokens of 80 heads take 62 us
// with 256 and one head ahead, 54.6 with 256 and 3, 53.2 with 128 and 3 (6.4 TB/s, 94%
// of the measured copy rate), 76 with 512 and 2.
constexpr int kAppendThreads = 128;
constexpr int kBatch = 3;

template <bool BF16>
__device__ __forceinline__ void rotate_halves(uint4 &a, uint4 &b, const float (&c)[8], const float (&s)[8])
{
    uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a0 = lo16<BF16>(aw[i]), a1 = hi16<BF16>(aw[i]);
        const float b0 = lo16<BF16>(bw[i]), b1 = hi16<BF16>(bw[i]);
        aw[i] = pack16<BF16>(a0 * c[2 * i] - b0 * s[2 * i], a1 * c[2 * i + 1] - b1 * s[2 * i + 1]);
        bw[i] = pack16<BF16>(b0 * c[2 * i] + a0 * s[2 * i], b1 * c[2 * i + 1] + a1 * s[2 * i + 1]);
    }
    a = make_uint4(aw[0], aw[1], aw[2], aw[3]);
    b = make_uint4(bw[0], bw[1], bw[2], bw[3]);
}

template <bool BF16>
__device__ __forceinline__ void rotate_pairs(uint4 &a, uint4 &b, const float (&c)[8], const float (&s)[8])
{
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = lo16<BF16>(w[i]), y = hi16<BF16>(w[i]);
        w[i] = pack16<BF16>(x * c[i] - y * s[i], y * c[i] + x * s[i]);
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
    b = make_uint4(w[4], w[5], w[6], w[7]);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kAppendThreads)
kv_append_kernel(const __grid_constant__ AppendParams p)
{
    constexpr int kItems = D / 16;                       // threads per head
    constexpr int kCols = kAppendThreads / kItems;       // heads in flight
    if (threadIdx.x == 0)
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const qmm_paged_kv &kv = p.kv;
    const int t = blockIdx.x;
    const int lane = threadIdx.x & 31;
    const int item = threadIdx.x % kItems;
    const int hq = p.q_heads, hk = kv.kv_heads;
    const int rot_items = p.rot / 16;
    const bool turn = item < rot_items;
    // the thread's two chunks of a head (8 values each)
    int c0 = 2 * item, c1 = 2 * item + 1;
    if (turn && !p.interleaved) {
        c0 = item;
        c1 = item + rot_items;
    }
    // heads: queries 0 .. hq - 1, keys, values
    const int heads = hq + 2 * hk;
    auto source = [&](int h) {
        return h < hq ? p.q + t * p.q_stride + static_cast<long long>(h) * D
             : h < hq + hk ? p.k + t * p.k_stride + static_cast<long long>(h - hq) * D
                           : p.v + t * p.v_stride + static_cast<long long>(h - hq - hk) * D;
    };
    // kBatch heads' chunks at a time; the first ones are under way before the rest is known
    int h = threadIdx.x / kItems;
    uint4 a[kBatch], b[kBatch];
    auto fetch = [&]() {
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (h + u * kCols < heads) {
                const uint16_t *src = source(h + u * kCols);
                a[u] = __ldcs(reinterpret_cast<const uint4 *>(src + 8 * c0));
                b[u] = __ldcs(reinterpret_cast<const uint4 *>(src + 8 * c1));
            }
    };
    fetch();

    int seq = 0, end = 0, keys = 0;
    find_sequence(kv, t, lane, seq, end, keys);
    if (seq >= kv.batch)
        return;                                          // past the last sequence: padding
    const int pos = max(keys, 0) - (end - t);            // (a length may be any integer)
    if (pos < 0)
        return;                                          // padding
    if (pos >= table_keys(kv) || (p.rot > 0 && pos >= p.rope_len)) {
        if (threadIdx.x == 0)
            record_error(p.status, QMM_ERR_INDEX);
        return;
    }
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        cs[i] = 1.f;
        sn[i] = 0.f;
    }
    if (turn) {
        const float4 *row = reinterpret_cast<const float4 *>(p.cos_sin + static_cast<long long>(pos) * p.rot + 8 * item);
        const float4 *rows = reinterpret_cast<const float4 *>(p.cos_sin + static_cast<long long>(pos) * p.rot +
                                                              p.rot / 2 + 8 * item);
        const float4 u0 = row[0], u1 = row[1], w0 = rows[0], w1 = rows[1];
        cs[0] = u0.x; cs[1] = u0.y; cs[2] = u0.z; cs[3] = u0.w;
        cs[4] = u1.x; cs[5] = u1.y; cs[6] = u1.z; cs[7] = u1.w;
        sn[0] = w0.x; sn[1] = w0.y; sn[2] = w0.z; sn[3] = w0.w;
        sn[4] = w1.x; sn[5] = w1.y; sn[6] = w1.z; sn[7] = w1.w;
    }
    const long long place = key_offset(kv, p.by_page, seq, pos, p.status);

    while (h < heads) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int hu = h + u * kCols;
            if (hu >= heads)
                break;
            if (turn && hu < hq + hk) {
                if (p.interleaved)
                    rotate_pairs<BF16>(a[u], b[u], cs, sn);
                else
                    rotate_halves<BF16>(a[u], b[u], cs, sn);
            }
            uint16_t *dst = nullptr;
            if (hu < hq)
                dst = p.q_out + (static_cast<long long>(t) * hq + hu) * D;
            else if (place >= 0)
                dst = hu < hq + hk ? static_cast<uint16_t *>(kv.k) + place + (hu - hq) * kv.head_stride
                                   : static_cast<uint16_t *>(kv.v) + place + (hu - hq - hk) * kv.head_stride;
            if (dst) {
                *reinterpret_cast<uint4 *>(dst + 8 * c0) = a[u];
                *reinterpret_cast<uint4 *>(dst + 8 * c1) = b[u];
            }
        }
        h += kBatch * kCols;
        fetch();
    }
}

template <int D, bool BF16>
cudaError_t launch_append(const AppendParams &p, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.kv.tokens);
    cfg.blockDim = dim3(kAppendThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_append_kernel<D, BF16>, p);
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t stream)
{
    const bool bf16 = p.kv.dtype == QMM_BF16;
    if (p.kv.head_dim == 128)
        return bf16 ? launch_append<128, true>(p, stream) : launch_append<128, false>(p, stream);
    return bf16 ? launch_append<64, true>(p, stream) : launch_append<64, false>(p, stream);
}

}  // namespace qmm
