// attn_rows.cuh -- how a block of few query rows ends (attn_decode.cu, kv4_decode.cu): its
// warps' results meet, and go to the output, to the cluster's other blocks or to scratch.
#pragma once

#include "paged.cuh"

namespace qmm {

namespace {

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

// The warps' unnormalized outputs lie in shared memory, [warp][ROWS][L::kPitch] from its
// start, their maxima and sums [warp][ROWS][2] at L::kOffMl, with a barrier after them.  A
// cluster's blocks send each other their parts (L::kOffIn, L::kOffInMl).  True: the item was
// the cluster's, and the block is done.
template <class L, int D, bool BF16, int WARPS, int ROWS>
__device__ __forceinline__ bool finish_rows(const AttnParams &p, const Segment &sg, uint8_t *smem)
{
    constexpr int kThreads = 32 * WARPS;
    const RowTile &r = sg.r;
    const int tid = threadIdx.x;
    const uint32_t sbase = smem_u32(smem);
    const float *wo = reinterpret_cast<const float *>(smem), *wml = reinterpret_cast<const float *>(smem + L::kOffMl);
    const int rank = blockIdx.x % p.cluster, log2_blocks = 31 - __clz(p.cluster);
    if (WARPS > 1 && p.cluster > 1) {
        cluster_wait();      // every block of the cluster has started
        // the block's maxima and sums of all rows to every block
        for (int e = tid; e < r.rows << log2_blocks; e += kThreads) {
            const int row = e >> log2_blocks;
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w)
                m = fmaxf(m, wml[(w * ROWS + row) * 2]);
            const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int w = 0; w < WARPS; ++w)
                l = fmaf(ex2(wml[(w * ROWS + row) * 2] - base), wml[(w * ROWS + row) * 2 + 1], l);
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
    for (int e = tid; e < r.rows * (D / 4); e += kThreads) {
        const int row = e / (D / 4), c = 4 * (e % (D / 4));
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
            m = fmaxf(m, wml[(w * ROWS + row) * 2]);
        const float base = m == -INFINITY ? 0.f : m;
        float l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float2 ml = *reinterpret_cast<const float2 *>(wml + (w * ROWS + row) * 2);
            const float a = ex2(ml.x - base);
            const float4 v = *reinterpret_cast<const float4 *>(wo + (w * ROWS + row) * L::kPitch + c);
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
        for (int i = tid; i < (r.rows * (D / 4)) >> log2_blocks; i += kThreads) {
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
        return true;
    }
    return false;
}

}  // namespace

}  // namespace qmm
