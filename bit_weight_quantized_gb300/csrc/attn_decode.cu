// attn_decode.cu -- attention over the paged cache for few query rows per key head
// (single tokens, short drafts): at most 16 rows (token, query head of the key
// head) per work item, which one m16 matrix-instruction tile holds.
//
//   s_j = scale <q, K_j>,  out = sum_j 2^(s_j' - m) V_j / sum_j 2^(s_j' - m),  s' = s log2(e)
//
// Bound by reading K and V once from HBM: every key costs 4 D bytes and at most
// 16 * 4 D flops, far below the tensor cores' ratio, so mma.sync is enough and the
// work is to keep reads in flight.  Each of a block's warps walks its own 16 keys
// (D = 64: 32) of every unit with its own ring of asynchronous copies (8 KB of K and V
// a stage), running maximum, sum and 16 x D fp32 output in registers: no barrier and
// no exchange between warps until the segment ends, when their results meet in shared
// memory.  Two blocks of four warps, or one of eight, per SM keep 128 KB in flight.
//
// Long axes are split over all blocks (find_share) and joined by a second kernel
// (attn.cu).  Short ones, where that kernel's 3.5 us would count, go to a cluster of
// up to eight blocks per item, each of which sends the others their share of its part to
// join, from shared memory to shared memory; blocks of eight warps halve its walk where
// an SM is free for each.  One token over 517 keys: 5.2 us.
//
// The running maximum is replaced only when it grows by more than 2^8 (the scale
// factors stay within fp32 and fp16 range either way), so the output is rescaled
// a few times per segment rather than in every tile: a published refinement of the running
// softmax; the bound is this file's, by the fp16 range below.  fp16 weights are scaled by
// 2^7: 2^(s' - m + 7) <= 2^15 stays finite and weights down to 2^-21 of the maximum
// keep all their bits (fp16 loses bits below 2^-14).
#include <atomic>

#include "paged.cuh"

namespace qmm {

namespace {

constexpr float kGrow = 8.f;                         // log2 of the growth that replaces the maximum

template <int D, int WARPS>
struct DecLayout {
    static constexpr int kWarpKeys = decode_keys(D, 4) / 4;               // a warp's keys of a unit
    static constexpr int kKeys = decode_keys(D, WARPS);                   // keys per unit
    static constexpr int kTile = kWarpKeys * D * 2;                       // their K or V, 4 KB
    static constexpr int kStages = 3;                                     // 24 KB of rings per warp
    static constexpr int kWarpBytes = kStages * 2 * kTile;
    static constexpr int kOffQ = WARPS * kWarpBytes;
    // what the cluster's blocks send this one: [value / 4 / blocks][block] four values,
    // [row][block] maximum and sum
    static constexpr int kOffIn = kOffQ + kDecodeRows * D * 2;
    static constexpr int kOffInMl = kOffIn + kDecodeRows * D * 4;
    static constexpr int kBytes = WARPS == 1 ? kOffIn : kOffInMl + kDecodeRows * kMaxCluster * 8;   // (one warp: no clusters)
    static constexpr int kPitch = D + 8;                                  // floats per row of a warp's output
    static constexpr int kOffMl = WARPS * kDecodeRows * kPitch * 4;   // the warps' maxima and sums
    static_assert(kOffMl + WARPS * kDecodeRows * 8 <= kOffQ, "the warps' outputs reuse the rings");
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <bool BF16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
            "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        mma_f16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
}

// Shared-memory byte of 16-byte chunk c of row r in a tile of D-value rows: chunks
// are permuted by the row so that eight rows of one chunk column (one ldmatrix
// matrix) lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t tile_addr(int r, int c)
{
    return static_cast<uint32_t>(r * D * 2 + ((c ^ (r & 7)) << 4));
}

// A shared-memory address of this block, in block `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, int rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void peer_store2(uint32_t addr, float a, float b)
{
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}

__device__ __forceinline__ void peer_store4(uint32_t addr, const float4 &v)
{
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// WARPS = 4: two blocks per SM; 8: one, for clusters where every block has an SM; 1:
// seven, for many short items.
template <int D, bool BF16, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WARPS == 4 ? kDecodeBlocksPerSm : WARPS == 8 ? 1 : kNarrowBlocksPerSm)
attn_decode_kernel(const __grid_constant__ AttnParams p)
{
    using L = DecLayout<D, WARPS>;
    constexpr int kDecThreads = 32 * WARPS;
    constexpr int kChunks = D / 8;                 // 16-byte chunks per row
    constexpr int kRowsPerCopy = 32 / kChunks;     // rows one warp-wide copy covers
    constexpr int kKeys = L::kKeys, kWarpKeys = L::kWarpKeys, kCopies = kWarpKeys / kRowsPerCopy;
    constexpr int kSub = kWarpKeys / 16;           // 16-key steps of the matrix instructions per tile
    constexpr float kShift = BF16 ? 0.f : 7.f;

    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Share share;
    __shared__ long long red[WARPS];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    if (tid == 0)
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (WARPS > 1 && p.cluster > 1)
        cluster_arrive();   // (waited for before anything is sent to another block)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    find_share<kKeys, kDecodeSetup, kDecThreads>(p, red, &share);

    const uint32_t sbase = smem_u32(smem);
    const uint32_t ring = sbase + warp * L::kWarpBytes;
    const uint32_t qs = sbase + L::kOffQ;
    // the lane's row and chunk in a warp-wide copy
    const int crow = lane / kChunks, cchunk = lane % kChunks;
    // its ldmatrix row and chunk: K (keys as the n index), V (transposed)
    const int krow = (lane & 7) + ((lane >> 4) << 3), kch = (lane >> 3) & 1;
    const int vrow = lane & 15, vch = lane >> 4;

    if (!p.whole && tid == 0)
        p.meta[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);

    Walk<kKeys, kDecodeSetup> walk;
    walk.begin(share);
    Segment sg;
    bool more = p.whole ? share.end > 0 : walk.next(p, sg);
    if (p.whole && more) {   // the whole item; a cluster's blocks take a stretch each
        const int rank = blockIdx.x % p.cluster, all = share.r.units;
        sg.r = share.r;
        sg.h = share.h;
        sg.start = 0;
        sg.off = rank * all / p.cluster;
        sg.units = (rank + 1) * all / p.cluster - sg.off;
    }
    if (WARPS > 1 && !more && p.cluster > 1)
        cluster_wait();
    for (; more; more = !p.whole && walk.next(p, sg)) {
        const RowTile &r = sg.r;
        const uint16_t *kbase = static_cast<const uint16_t *>(p.kv.k) + sg.h * p.kv.head_stride;
        const uint16_t *vbase = static_cast<const uint16_t *>(p.kv.v) + sg.h * p.kv.head_stride;
        const int key0 = (r.unit0 + sg.off) * kKeys + warp * kWarpKeys;   // the warp's first key

        // Where tile j lies: where a tile's keys share a page (p.same_page), the offset of
        // the lane's first row; else that of row `lane`.  -1: nothing is read.  The page is
        // looked up one tile ahead and not looked at before the tile is loaded: the warp
        // would wait for the table's entry here.
        auto key_of = [&](int j) { return key0 + j * kKeys + (p.same_page ? 0 : lane % kWarpKeys); };
        auto reads = [&](int j) {
            const int key = key_of(j);
            return j < sg.units && key < r.hi && (p.same_page ? key + kWarpKeys : key + 1) > r.lo;
        };
        auto look_up = [&](int j) -> int {
            return reads(j) ? p.kv.block_table[static_cast<long long>(r.b) * p.kv.blocks + p.by_page(key_of(j))] : 0;
        };
        auto place = [&](int j, int page) -> long long {
            if (!reads(j))
                return -1;
            if (page < 0 || page >= p.kv.num_pages) {
                record_error(p.status, QMM_ERR_INDEX);
                return -1;
            }
            const int key = key_of(j), slot = key - p.by_page(key) * p.kv.page_size;
            return page * p.kv.page_stride + (slot + (p.same_page ? crow : 0)) * p.kv.slot_stride;
        };
        auto load = [&](int j, long long off) {
            const uint32_t dst = ring + (j % L::kStages) * (2 * L::kTile);
            if (p.same_page) {
                const int kb = key0 + j * kKeys;
                const bool inside = off >= 0 && kb >= r.lo && kb + kWarpKeys <= r.hi;
                const long long step = kRowsPerCopy * p.kv.slot_stride;
                long long e = off + cchunk * 8;
#pragma unroll
                for (int c = 0; c < kCopies; ++c) {
                    const int row = c * kRowsPerCopy + crow, key = kb + row;
                    const bool ok = inside || (off >= 0 && key >= r.lo && key < r.hi);
                    cp_async16_or_zero(dst + tile_addr<D>(row, cchunk), ok ? kbase + e : p.q, ok);
                    cp_async16_or_zero(dst + L::kTile + tile_addr<D>(row, cchunk), ok ? vbase + e : p.q, ok);
                    e += step;
                }
                return;
            }
#pragma unroll
            for (int c = 0; c < kCopies; ++c) {
                const int row = c * kRowsPerCopy + crow;
                const long long o = __shfl_sync(0xffffffffu, off, row);
                const bool ok = o >= 0;
                const long long e = o + cchunk * 8;
                cp_async16_or_zero(dst + tile_addr<D>(row, cchunk), ok ? kbase + e : p.q, ok);
                cp_async16_or_zero(dst + L::kTile + tile_addr<D>(row, cchunk), ok ? vbase + e : p.q, ok);
            }
        };

        int page[L::kStages - 1];
#pragma unroll
        for (int j = 0; j < L::kStages - 1; ++j)
            page[j] = look_up(j);
        int ahead = look_up(L::kStages - 1);
        // queries: 16 rows, zero past the tile
        for (int e = tid; e < kDecodeRows * kChunks; e += kDecThreads) {
            const int row = e / kChunks, c = e % kChunks, rr = r.row0 + row, tok = p.by_group(rr);
            const bool in = row < r.rows;
            const uint16_t *src = p.q;
            if (in)
                src += (r.t0 + tok) * p.q_stride + static_cast<long long>(sg.h * p.group + rr - tok * p.group) * D + 8 * c;
            cp_async16_or_zero(qs + tile_addr<D>(row, c), src, in);
        }
        cp_async_commit();
#pragma unroll
        for (int j = 0; j < L::kStages - 1; ++j) {
            if (j < sg.units)
                load(j, place(j, page[j]));
            cp_async_commit();
        }

        // the queries have landed (the copies after them are still under way); to
        // registers in fragment order
        cp_async_wait_group<L::kStages - 1>();
        __syncthreads();
        uint32_t qf[D / 16][4];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
            ldsm4(qf[kk], qs + tile_addr<D>(lane & 15, 2 * kk + (lane >> 4)));

        const int2 see0 = row_keys(p, r, r.row0 + g), see1 = row_keys(p, r, r.row0 + g + 8);
        // keys that every row of the tile sees (rows past the tile do not count)
        const int2 sa = row_keys(p, r, r.row0), sz = row_keys(p, r, r.row0 + r.rows - 1);
        const int all_lo = sz.x, all_hi = sa.y;

        float o[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[n][e] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

#pragma unroll 1
        for (int j = 0; j < sg.units; ++j) {
            if (j + L::kStages - 1 < sg.units)
                load(j + L::kStages - 1, place(j + L::kStages - 1, ahead));
            cp_async_commit();
            ahead = look_up(j + L::kStages);
            cp_async_wait_group<L::kStages - 1>();
            __syncwarp();
            const int kb = key0 + j * kKeys;
            if (kb < r.hi && kb + kWarpKeys > r.lo) {
                const uint32_t ks = ring + (j % L::kStages) * (2 * L::kTile), vs = ks + L::kTile;
                float s[2 * kSub][4];
#pragma unroll
                for (int n = 0; n < 2 * kSub; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[n][e] = 0.f;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int u = 0; u < kSub; ++u) {
                        uint32_t kf[4];
                        ldsm4(kf, ks + tile_addr<D>(16 * u + krow, 2 * kk + kch));
                        mma16<BF16>(s[2 * u], qf[kk], kf[0], kf[1]);
                        mma16<BF16>(s[2 * u + 1], qf[kk], kf[2], kf[3]);
                    }
                if (kb < all_lo || kb + kWarpKeys - 1 > all_hi) {
#pragma unroll
                    for (int n = 0; n < 2 * kSub; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int key = kb + 8 * n + 2 * t + e;
                            if (key < see0.x || key > see0.y)
                                s[n][e] = -INFINITY;
                            if (key < see1.x || key > see1.y)
                                s[n][2 + e] = -INFINITY;
                        }
                }
                float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
                for (int n = 0; n < 2 * kSub; ++n) {
                    x0 = fmaxf(x0, fmaxf(s[n][0], s[n][1]));
                    x1 = fmaxf(x1, fmaxf(s[n][2], s[n][3]));
                }
                x0 *= p.scale_log2;
                x1 *= p.scale_log2;
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
                const bool up0 = x0 > m0 + kGrow, up1 = x1 > m1 + kGrow;
                if (__any_sync(0xffffffffu, up0 || up1)) {
                    const float a0 = up0 ? ex2(m0 - x0) : 1.f, a1 = up1 ? ex2(m1 - x1) : 1.f;
                    m0 = up0 ? x0 : m0;
                    m1 = up1 ? x1 : m1;
                    l0 *= a0;
                    l1 *= a1;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[n][0] *= a0;
                        o[n][1] *= a0;
                        o[n][2] *= a1;
                        o[n][3] *= a1;
                    }
                }
                const float n0 = kShift - (m0 == -INFINITY ? 0.f : m0), n1 = kShift - (m1 == -INFINITY ? 0.f : m1);
                uint32_t pf[kSub][4];
#pragma unroll
                for (int n = 0; n < 2 * kSub; ++n) {
                    const float p0 = ex2(fmaf(s[n][0], p.scale_log2, n0)), p1 = ex2(fmaf(s[n][1], p.scale_log2, n0));
                    const float p2 = ex2(fmaf(s[n][2], p.scale_log2, n1)), p3 = ex2(fmaf(s[n][3], p.scale_log2, n1));
                    l0 += p0 + p1;
                    l1 += p2 + p3;
                    pf[n / 2][2 * (n & 1)] = pack16<BF16>(p0, p1);
                    pf[n / 2][2 * (n & 1) + 1] = pack16<BF16>(p2, p3);
                }
#pragma unroll
                for (int u = 0; u < kSub; ++u)
#pragma unroll
                    for (int n = 0; n < D / 16; ++n) {
                        uint32_t vf[4];
                        ldsm4_t(vf, vs + tile_addr<D>(16 * u + vrow, 2 * n + vch));
                        mma16<BF16>(o[2 * n], pf[u], vf[0], vf[1]);
                        mma16<BF16>(o[2 * n + 1], pf[u], vf[2], vf[3]);
                    }
            }
            __syncwarp();   // every lane has read the slot before it is filled again
        }
        cp_async_wait_group<0>();
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, d);
            l1 += __shfl_xor_sync(0xffffffffu, l1, d);
        }

        // the warps' maxima, sums and outputs meet in shared memory (over the rings)
        __syncthreads();
        float *wo = reinterpret_cast<float *>(smem);
        float *wml = reinterpret_cast<float *>(smem + L::kOffMl);
        {
            float *w0 = wo + (warp * kDecodeRows + g) * L::kPitch, *w1 = w0 + 8 * L::kPitch;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
                *reinterpret_cast<float2 *>(w0 + 8 * n + 2 * t) = make_float2(o[n][0], o[n][1]);
                *reinterpret_cast<float2 *>(w1 + 8 * n + 2 * t) = make_float2(o[n][2], o[n][3]);
            }
            if (t == 0) {
                *reinterpret_cast<float2 *>(wml + (warp * kDecodeRows + g) * 2) = make_float2(m0, l0);
                *reinterpret_cast<float2 *>(wml + (warp * kDecodeRows + g + 8) * 2) = make_float2(m1, l1);
            }
        }
        __syncthreads();
        const int rank = blockIdx.x % p.cluster, log2_blocks = 31 - __clz(p.cluster);
        if (WARPS > 1 && p.cluster > 1) {
            cluster_wait();      // every block of the cluster has started
            // the block's maxima and sums of all rows to every block
            for (int e = tid; e < r.rows << log2_blocks; e += kDecThreads) {
                const int row = e >> log2_blocks;
                float m = -INFINITY, l = 0.f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w)
                    m = fmaxf(m, wml[(w * kDecodeRows + row) * 2]);
                const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
                for (int w = 0; w < WARPS; ++w)
                    l = fmaf(ex2(wml[(w * kDecodeRows + row) * 2] - base), wml[(w * kDecodeRows + row) * 2 + 1], l);
                peer_store2(peer_addr(sbase + L::kOffInMl + (row * p.cluster + rank) * 8, e & (p.cluster - 1)), m, l);
            }
        }
        const bool whole = is_whole(sg);
        const int slot = part_slot(sg);
        // four finished values of a row to the output
        auto store = [&](int row, int c, float m, float l, const float4 &acc) {
            const int rr = r.row0 + row, tok = p.by_group(rr);
            const long long at = static_cast<long long>(r.t0 + tok) * p.q_heads + sg.h * p.group + rr - tok * p.group;
            const float inv = row_inverse(l);
            *reinterpret_cast<uint2 *>(p.out + at * D + c) =
                make_uint2(pack16<BF16>(acc.x * inv, acc.y * inv), pack16<BF16>(acc.z * inv, acc.w * inv));
            if (p.lse && c == 0)
                p.lse[at] = row_log_sum<BF16>(m, l);
        };
        for (int e = tid; e < r.rows * (D / 4); e += kDecThreads) {
            const int row = e / (D / 4), c = 4 * (e % (D / 4));
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < WARPS; ++w)
                m = fmaxf(m, wml[(w * kDecodeRows + row) * 2]);
            const float base = m == -INFINITY ? 0.f : m;
            float l = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float2 ml = *reinterpret_cast<const float2 *>(wml + (w * kDecodeRows + row) * 2);
                const float a = ex2(ml.x - base);
                const float4 v = *reinterpret_cast<const float4 *>(wo + (w * kDecodeRows + row) * L::kPitch + c);
                l = fmaf(a, ml.y, l);
                acc.x = fmaf(a, v.x, acc.x);
                acc.y = fmaf(a, v.y, acc.y);
                acc.z = fmaf(a, v.z, acc.z);
                acc.w = fmaf(a, v.w, acc.w);
            }
            if (WARPS > 1 && p.cluster > 1) {   // four values to the block that joins them
                peer_store4(peer_addr(sbase + L::kOffIn + ((e >> log2_blocks) * p.cluster + rank) * 16, e & (p.cluster - 1)), acc);
            } else if (whole) {
                store(row, c, m, l, acc);
            } else {
                *reinterpret_cast<float4 *>(p.part_o + (static_cast<long long>(slot) * kDecodeRows + row) * D + c) = acc;
                if (c == 0)
                    *reinterpret_cast<float2 *>(p.part_ml + (static_cast<long long>(slot) * kDecodeRows + row) * 2) =
                        make_float2(m, l);
            }
        }
        if (WARPS > 1 && p.cluster > 1) {
            // each block joins its share of the values.  They have been sent to it: reading
            // them from the others takes a second meeting, before which no block may leave,
            // and 1 us more.
            cluster_arrive();
            cluster_wait();
            for (int i = tid; i < (r.rows * (D / 4)) >> log2_blocks; i += kDecThreads) {
                const int e = (i << log2_blocks) + rank, row = e / (D / 4), c = 4 * (e % (D / 4));
                const float4 *v = reinterpret_cast<const float4 *>(smem + L::kOffIn) + (i << log2_blocks);
                const float2 *ml = reinterpret_cast<const float2 *>(smem + L::kOffInMl) + (row << log2_blocks);
                float m = -INFINITY, l = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int b = 0; b < p.cluster; ++b)
                    m = fmaxf(m, ml[b].x);
                const float base = m == -INFINITY ? 0.f : m;
                for (int b = 0; b < p.cluster; ++b) {
                    const float w = ex2(ml[b].x - base);
                    l = fmaf(w, ml[b].y, l);
                    acc.x = fmaf(w, v[b].x, acc.x);
                    acc.y = fmaf(w, v[b].y, acc.y);
                    acc.z = fmaf(w, v[b].z, acc.z);
                    acc.w = fmaf(w, v[b].w, acc.w);
                }
                store(row, c, m, l, acc);
            }
            return;
        }
        if (tid == 0 && is_last_part(sg))
            write_meta<kDecodeSetup>(p, sg, share.chunk);
        __syncthreads();   // the rings and the query tile are free again
    }
}

template <int D, bool BF16, int WARPS>
cudaError_t decode_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&attr)[2], int grid, int cluster,
                          cudaStream_t stream)
{
    constexpr int smem = DecLayout<D, WARPS>::kBytes;
    static SmemLimit limit;
    if (const cudaError_t e = ensure_smem_limit(limit, attn_decode_kernel<D, BF16, WARPS>, smem, true); e != cudaSuccess)
        return e;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(32 * WARPS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaSuccess;
}

template <int D, bool BF16, int WARPS>
cudaError_t launch_decode_attn(const AttnParams &p, int grid, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    if (const cudaError_t e = decode_config<D, BF16, WARPS>(cfg, attr, grid, p.cluster, stream); e != cudaSuccess)
        return e;
    return cudaLaunchKernelEx(&cfg, attn_decode_kernel<D, BF16, WARPS>, p);
}

// Clusters of 2, 4 or 8 blocks that run at once on the current device: fewer than its
// blocks' number would give, since a cluster lies in one part of the device.
template <int D, bool BF16, int WARPS>
int active_clusters(int cluster)
{
    static std::atomic<int> known[64][4] = {};   // + 1; per device and log2 of the size
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return 0;
    std::atomic<int> &k = known[dev][cluster == 2 ? 1 : cluster == 4 ? 2 : 3];
    if ((n = k.load(std::memory_order_relaxed)) > 0)
        return n - 1;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    if (decode_config<D, BF16, WARPS>(cfg, attr, cluster, cluster, nullptr) != cudaSuccess)
        return 0;
    cfg.attrs = attr + 1;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, attn_decode_kernel<D, BF16, WARPS>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    k.store(n + 1, std::memory_order_relaxed);
    return n;
}

template <int D, bool BF16>
cudaError_t launch_decode_width(const AttnParams &p, int grid, cudaStream_t stream)
{
    return p.warps == 8   ? launch_decode_attn<D, BF16, 8>(p, grid, stream)
           : p.warps == 4 ? launch_decode_attn<D, BF16, 4>(p, grid, stream)
                          : launch_decode_attn<D, BF16, 1>(p, grid, stream);
}

}  // namespace

cudaError_t launch_attn_decode(const AttnParams &p, int grid, cudaStream_t stream)
{
    const bool bf16 = p.kv.dtype == QMM_BF16;
    if (p.kv.head_dim == 128)
        return bf16 ? launch_decode_width<128, true>(p, grid, stream) : launch_decode_width<128, false>(p, grid, stream);
    return bf16 ? launch_decode_width<64, true>(p, grid, stream) : launch_decode_width<64, false>(p, grid, stream);
}

int attn_decode_clusters(int head_dim, bool bf16, int warps, int cluster)
{
    if (head_dim == 128)
        return warps == 8 ? (bf16 ? active_clusters<128, true, 8>(cluster) : active_clusters<128, false, 8>(cluster))
                          : (bf16 ? active_clusters<128, true, 4>(cluster) : active_clusters<128, false, 4>(cluster));
    return warps == 8 ? (bf16 ? active_clusters<64, true, 8>(cluster) : active_clusters<64, false, 8>(cluster))
                      : (bf16 ? active_clusters<64, true, 4>(cluster) : active_clusters<64, false, 4>(cluster));
}

}  // namespace qmm
