// kv4_decode.cu -- attention over the 4-bit paged cache for few query rows per key head:
// at most 16 rows (token, query head of the key head) per work item.
//
//   K_j = (c_j - z) s per 64 values, likewise V_j:
//   S_j = sum_g s_jg (sum_d q_d c_jd - z_jg sum_d q_d),  O = sum_j p_j s_jg (c_jd - z_jg)
//
// The codes themselves are the matrix instructions' operands; scales and zeros meet the
// scores and the weights, of which there are D times fewer.  A code in the low four bits of
// an fp16 pattern is the (subnormal) number c 2^-24, in the next four c 2^-20, both exact: a
// word of eight codes becomes four operand words by a shift and four masks.  Which d a
// place along an operand's axis stands for is free, so the queries are loaded in that
// order, those against c 2^-20 scaled by 2^-4.  The tile is turned over (keys are the rows
// of the scores' product, d those of the output's), so that 8 query rows, the most that a
// single token of most models has per key head, fill an instruction: as columns.
//
// A product with a subnormal operand is aligned by its exponent field, so that sums keep
// 2^-14 of a step s instead of fp32's precision: measured 2^-15 of a weight times s, where
// the cache's own error is s / 2.  (Codes as 64 + c, normal numbers, would take 7
// instructions for 8 codes instead of 5.)
//
// Queries are scaled per row by a power of two to below 2^15 and are then fp16 (bf16 has
// 8 bits, so only values 2^-25 times the row's largest lose any).  A weight times its V
// scale is rounded once to fp16, 2^-12 relative, times a power of two of its row and group that
// follows the largest such product so far (2^7 to 2^16 then), as the maximum follows the scores:
// what a key's large values take from the others' bits depends on its weight, in the group that
// holds them and the rows that see it.  (One power of two per warp, from the largest scale, left
// nothing of keys 2^-32 times that scale, whatever its weight; 64 sequences 51.4 us with it, 52.4.)
// That the zeros' share is subtracted by the same rounded weights comes from one more product, of the zeros.
//
// Bound by latency, with no unit full (DRAM 50%, issue 50%, logic pipe 51%, tensor 19% of a launch, of
// which start and join take a third): a warp's tile goes from scores to maximum, weights and output in
// order, with four warps a scheduler to cover it.  The loop takes some 307 instructions a warp for 16
// keys of 128, 2176 bytes, which the copy rate brings in 372 issue slots.  64 sequences of 300 to 4096
// keys, 8 key heads: 52.4 us (copies alone 36, the first form of this kernel 58.5); one token over 131072
// keys 44.7.  Each of a block's warps walks its own keys with its own ring of asynchronous copies,
// maximum, sum and output, as in attn_decode.cu, whose split, clusters and end this has.
#include <atomic>
#include <cuda_fp16.h>

#include "attn_rows.cuh"
#include "kv4.cuh"

namespace qmm {

namespace {

constexpr float kGrow = 8.f;                         // log2 of the growth that replaces the maximum

template <int D, int WARPS, int NB>
struct Layout {
    static constexpr int kRows = 8 * NB;
    static constexpr int kWarpKeys = kv4_keys(D, 1);                      // a warp's keys of a unit
    static constexpr int kKeys = kv4_keys(D, WARPS);
    static constexpr int kRow = D / 2, kScaleRow = D / 16;                // bytes of a key's codes, and of both its scales
    static constexpr int kCodes = kWarpKeys * kRow;                       // 2 KB
    static constexpr int kStage = 2 * kCodes + kWarpKeys * kScaleRow;
    static constexpr int kStages = 3;
    static constexpr int kWarpBytes = kStages * kStage;
    // queries in operand order; per row minus its groups' sums and the factor of its scores
    static constexpr int kOffQ = WARPS * kWarpBytes;
    static constexpr int kOffRow = kOffQ + kRows * D * 2;
    static constexpr int kOffIn = kOffRow + kRows * 16;                   // clusters: what the other blocks send
    static constexpr int kOffInMl = kOffIn + kRows * D * 4;
    static constexpr int kBytes = kOffIn, kClusterBytes = kOffInMl + kRows * kMaxCluster * 8;
    static constexpr int kPitch = D + 8;
    static constexpr int kOffMl = WARPS * kRows * kPitch * 4;
    static_assert(kOffMl + WARPS * kRows * 8 <= kOffQ, "the warps' outputs reuse the rings");
};

// (plain loads: the compiler moves them between the waits, which are barriers to it)
__device__ __forceinline__ uint32_t lds32(const uint8_t *p) { return *reinterpret_cast<const uint32_t *>(p); }
__device__ __forceinline__ uint2 lds64(const uint8_t *p) { return *reinterpret_cast<const uint2 *>(p); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// An 8 x 8 matrix of 16-bit values, row g of it in lane group g: turned over.
__device__ __forceinline__ uint32_t transpose8(uint32_t v)
{
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}

// The key (row of a 16-key step, eight by eight) that index k of an operand's axis stands
// for: with it and the swizzle below, neither the K reads (keys k = 0 .. 3 or 4 .. 7 at once)
// nor the V reads (even or odd k) meet in a bank.
__device__ __forceinline__ int key_row(int k) { return (k >> 1 & 1) | ((k ^ k >> 2) & 1) << 1 | (k & 4) | (k & 8); }

// Byte of 16-byte chunk c of row r of a tile of codes.
template <int D>
__device__ __forceinline__ uint32_t code_addr(int r, int c)
{
    return static_cast<uint32_t>(r * (D / 2) + ((D == 128 ? c ^ (r & 2) : c) << 4));
}

// Both halves of a word as numbers: 16-bit floats of the type, or fp16.
template <bool BF16>
__device__ __forceinline__ void halves(uint32_t w, float &lo, float &hi)
{
    if constexpr (BF16) {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xffff0000u);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        lo = f.x;
        hi = f.y;
    }
}

__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Column e of a group's output fragments, and of the zeros' share, times `by`.
__device__ __forceinline__ void scale_output(float (&o)[4][4], float (&oz)[4], int e, float by)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[i][e] *= by;
        o[i][2 + e] *= by;
    }
    oz[e] *= by;
    oz[2 + e] *= by;
}

template <int D, bool BF16, int WARPS, int NB>
__global__ void __launch_bounds__(32 * WARPS, kv4_blocks_per_sm(8 * NB, WARPS))
kv4_decode_kernel(const __grid_constant__ Kv4AttnParams p)
{
    using L = Layout<D, WARPS, NB>;
    constexpr int kThreads = 32 * WARPS, kKeys = L::kKeys, kWarpKeys = L::kWarpKeys, kRows = L::kRows;
    constexpr int kGroups = D / kKv4Group, kSteps = kWarpKeys / 16;
    constexpr int kChunks = D / 32;                    // 16-byte chunks of a key's codes
    constexpr int kRowsPerCopy = 32 / kChunks, kCopies = kWarpKeys / kRowsPerCopy;
    constexpr int kLook = kWarpKeys / 32;              // keys whose place a lane looks up, per tile
    // weights are 2^(s - m + 7), at most 2^15: times a V scale and f, they are rounded to fp16
    constexpr float kShift = 7.f;
    constexpr uint32_t kM0 = 0x000f000fu, kM1 = 0x00f000f0u, kMB = 0x00ff00ffu, kScaleBits = 0xfff0fff0u;
    constexpr int kMostF = 127 + 112;                  // f's exponent field at most: 2^15 times it is a number

    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Share share;
    __shared__ long long red[WARPS];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    if (tid == 0)
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (p.cluster > 1)
        cluster_arrive();   // (waited for before anything is sent to another block)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    find_share<kKeys, kDecodeSetup, kThreads, true>(p, red, &share);

    uint8_t *const ring = smem + warp * L::kWarpBytes, *const ring_end = ring + L::kWarpBytes;
    const int crow = lane / kChunks, cchunk = lane % kChunks;
    // the lane's places in a stage: K words of key g (of 16) and their scales, V words of keys
    // 2 t and 2 t + 1 and their zeros, the scales of key `lane`
    uint32_t at_k[kGroups], at_v[2][kGroups], at_z[2];
#pragma unroll
    for (int gr = 0; gr < kGroups; ++gr)
        at_k[gr] = code_addr<D>(key_row(g), 2 * gr + (t >> 1)) + 8 * (t & 1);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int gr = 0; gr < kGroups; ++gr)
            at_v[e][gr] = L::kCodes + code_addr<D>(key_row(2 * t + e), 2 * gr + (g >> 2)) + 4 * (g & 3);
        at_z[e] = 2 * L::kCodes + key_row(2 * t + e) * L::kScaleRow + (kGroups == 2 ? 4 : 0);
    }
    const uint32_t at_s = 2 * L::kCodes + key_row(g) * L::kScaleRow;

    if (!p.whole && tid == 0)
        p.meta[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);

    Walk<kKeys, kDecodeSetup, true> walk;
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
    if (!more && p.cluster > 1)
        cluster_wait();
    for (; more; more = !p.whole && walk.next(p, sg)) {
        const RowTile &r = sg.r;
        const int s_page = static_cast<int>(p.sc.page), s_slot = static_cast<int>(p.sc.slot);
        const uint8_t *kbase = static_cast<const uint8_t *>(p.kv.k) + sg.h * p.kv.head_stride + cchunk * 16;
        const uint8_t *vbase = static_cast<const uint8_t *>(p.kv.v) + sg.h * p.kv.head_stride + cchunk * 16;
        const uint16_t *sbase = p.sc.base + sg.h * p.sc.head;
        const int32_t *pages = p.kv.block_table + static_cast<long long>(r.b) * p.kv.blocks;
        // the warp's first place of tile j (places, not keys: see row_tile)
        const int place0 = sg.off * kKeys + warp * kWarpKeys;
        auto tile_place = [&](int j) { return place0 + j * kKeys; };
        // The places of the lane's keys of a tile (lane, lane + 32; slot -1: nobody sees it) are
        // looked up one tile ahead and not looked at before the tile is loaded: the warp would wait
        // for the table here.
        struct Look {
            int page[kLook], slot[kLook];
        };
        auto look_up = [&](int j) {
            Look k;
#pragma unroll
            for (int i = 0; i < kLook; ++i) {
                const int place = tile_place(j) + lane + 32 * i, key = place + (place < p.sinks ? 0 : r.lo), blk = p.by_page(key);
                const bool in = j < sg.units && place < r.hi;
                k.slot[i] = in ? key - blk * p.kv.page_size : -1;
                k.page[i] = in ? pages[blk] : 0;
            }
            return k;
        };
        auto load = [&](const Look &look, uint8_t *stage) {
            const uint32_t dst = smem_u32(stage);
            uint32_t off[kLook];                     // of the key's codes, in p.unit bytes
            bool all = true, good[kLook];
#pragma unroll
            for (int i = 0; i < kLook; ++i) {
                const int page = look.page[i], slot = look.slot[i];
                good[i] = slot >= 0;
                if (good[i] && static_cast<unsigned>(page) >= static_cast<unsigned>(p.kv.num_pages)) {
                    record_error(p.status, QMM_ERR_INDEX);
                    good[i] = false;
                }
                off[i] = good[i] ? page * p.page_units + slot * p.slot_units : ~0u;
                all = all && good[i];
                // (a key that nobody sees gets scales of zero; its codes do not matter)
                const uint16_t *src = sbase + static_cast<long long>(good[i] ? page : 0) * s_page + (good[i] ? slot * s_slot : 0);
                cp_async_small<L::kScaleRow>(dst + 2 * L::kCodes + (lane + 32 * i) * L::kScaleRow, src, good[i]);
            }
            const uint32_t to = dst + code_addr<D>(crow, cchunk);   // (its permutation has the period of a copy's rows)
            if (__all_sync(0xffffffffu, all)) {
#pragma unroll
                for (int c = 0; c < kCopies; ++c) {
                    const uint32_t o = __shfl_sync(0xffffffffu, off[c * kRowsPerCopy / 32], (c * kRowsPerCopy + crow) & 31);
                    cp_async16(to + c * kRowsPerCopy * L::kRow, kbase + static_cast<uint64_t>(o) * p.unit);
                    cp_async16(to + c * kRowsPerCopy * L::kRow + L::kCodes, vbase + static_cast<uint64_t>(o) * p.unit);
                }
                return;
            }
#pragma unroll 1
            for (int c = 0; c < kCopies; ++c) {
                const uint32_t o = __shfl_sync(0xffffffffu, kLook == 2 && c * kRowsPerCopy >= 32 ? off[kLook - 1] : off[0],
                                               (c * kRowsPerCopy + crow) & 31);
                const bool ok = o != ~0u;
                const uint64_t e = ok ? static_cast<uint64_t>(o) * p.unit : 0;
                cp_async16_or_zero(to + c * kRowsPerCopy * L::kRow, kbase + e, ok);
                cp_async16_or_zero(to + c * kRowsPerCopy * L::kRow + L::kCodes, vbase + e, ok);
            }
        };

        Look first[L::kStages - 1];
#pragma unroll
        for (int j = 0; j < L::kStages - 1; ++j)
            first[j] = look_up(j);
        Look ahead = look_up(L::kStages - 1);

        // Queries in operand order, eight values a thread: 16 bytes of a row, gone through by half a
        // warp (D = 64: a quarter).  By all warps, since code that runs once per segment has to be
        // fetched, at several cycles an instruction: every warp's own fragments, straight from
        // memory, took some 500 instructions.
        constexpr int kWords = D / 8, kItems = kRows * kWords;
        uint4 raw[(kItems + kThreads - 1) / kThreads];
#pragma unroll
        for (int i = 0; i * kThreads < kItems; ++i) {
            const int e = i * kThreads + tid, row = e / kWords, rr = r.row0 + row, tok = p.by_group(rr);
            raw[i] = make_uint4(0u, 0u, 0u, 0u);
            if (e < kItems && row < r.rows)
                raw[i] = *reinterpret_cast<const uint4 *>(p.q + (r.t0 + tok) * p.q_stride +
                                                          static_cast<long long>(sg.h * p.group + rr - tok * p.group) * D + 8 * (e % kWords));
        }
        uint8_t *wr = ring, *rd = ring;              // the stages written and read next
        auto next_stage = [&](uint8_t *a) { return a + L::kStage == ring_end ? ring : a + L::kStage; };
#pragma unroll 1
        for (int j = 0; j < L::kStages - 1; ++j) {
            if (j < sg.units)
                load(first[0], wr);
            cp_async_commit();
            wr = next_stage(wr);
#pragma unroll
            for (int i = 0; i + 1 < L::kStages - 1; ++i)
                first[i] = first[i + 1];
        }
#pragma unroll
        for (int i = 0; i * kThreads < kItems; ++i) {
            const int e = i * kThreads + tid;
            if (e >= kItems)                         // (whole warps)
                break;
            const uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
            float v[8], most = 0.f, sum = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[2 * k] = lo16<BF16>(x[k]);
                v[2 * k + 1] = hi16<BF16>(x[k]);
                most = fmaxf(most, fmaxf(fabsf(v[2 * k]), fabsf(v[2 * k + 1])));
            }
#pragma unroll
            for (int d = 1; d < kWords; d <<= 1)
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
            // a power of two that brings the largest to 2^14 .. 2^15 (exponents kept where both
            // it and its inverse with the codes' 2^24 are normal numbers)
            const uint32_t ex = min(max(__float_as_uint(most) >> 23, 15u), 243u);
            const float down = __uint_as_float((268u - ex) << 23);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[k] *= down;
                sum += v[k];
            }
#pragma unroll
            for (int d = 1; d < 8; d <<= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, d);
            *reinterpret_cast<uint4 *>(smem + L::kOffQ + 16 * e) =
                make_uint4(pack16<false>(v[0], v[4]), pack16<false>(v[2], v[6]), pack16<false>(v[1] * 0.0625f, v[5] * 0.0625f),
                           pack16<false>(v[3] * 0.0625f, v[7] * 0.0625f));
            float *rows = reinterpret_cast<float *>(smem + L::kOffRow) + 4 * (e / kWords);
            if (e % 8 == 0)                          // minus the group's sum, the scores' factor
                rows[e % kWords / 8] = -sum;
            if (e % kWords == 0)                     // (not zero, which times a hidden score, -infinity, is NaN)
                rows[2] = fmaxf(__uint_as_float((ex + 10u) << 23) * p.scale_log2, __uint_as_float(1));
        }
        __syncthreads();
        uint32_t qf[NB][kGroups][4][2];
        float qs[NB][kGroups][2], rowf[NB][2];       // of rows 2 t, 2 t + 1
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int gr = 0; gr < kGroups; ++gr)
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(smem + L::kOffQ + 16 * ((8 * nb + g) * kWords + 8 * gr + 2 * t + w));
                    qf[nb][gr][2 * w][0] = u.x;
                    qf[nb][gr][2 * w][1] = u.y;
                    qf[nb][gr][2 * w + 1][0] = u.z;
                    qf[nb][gr][2 * w + 1][1] = u.w;
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float4 u = reinterpret_cast<const float4 *>(smem + L::kOffRow)[8 * nb + 2 * t + e];
                qs[nb][0][e] = u.x;
                if (kGroups == 2)
                    qs[nb][kGroups - 1][e] = u.y;
                rowf[nb][e] = u.z;
            }
        }

        // places that the lane's rows see, and that every row of the tile sees (rows past the
        // tile do not count)
        int2 see[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                see[nb][e] = row_places(p, r, r.row0 + 8 * nb + 2 * t + e);
        const int all_lo = row_places(p, r, r.row0 + r.rows - 1).x, all_hi = row_places(p, r, r.row0).y;

        float o[NB][kGroups][4][4], oz[NB][kGroups][4];   // [tile of d][fragment]; the zeros' share
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int gr = 0; gr < kGroups; ++gr)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    oz[nb][gr][e] = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[nb][gr][i][e] = 0.f;
                }
        // kShift - the maximum, the score past which it is replaced (-infinity: there
        // is none yet), the sum; per group f, the power of two by which weights times V scales are taken
        float minus[NB][2], limit[NB][2], l[NB][2], f[NB][kGroups][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                minus[nb][e] = kShift;
                limit[nb][e] = -INFINITY;
                l[nb][e] = 0.f;
#pragma unroll
                for (int gr = 0; gr < kGroups; ++gr)
                    f[nb][gr][e] = __uint_as_float(kMostF << 23);
            }

#pragma unroll 1
        for (int j = 0; j < sg.units; ++j) {
            if (j + L::kStages - 1 < sg.units)
                load(ahead, wr);
            cp_async_commit();
            wr = next_stage(wr);
            ahead = look_up(j + L::kStages);
            cp_async_wait_group<L::kStages - 1>();
            __syncwarp();
            const int kb = tile_place(j);
            if (kb < r.hi) {
                // scores: rows are keys, columns query rows
                float s[kSteps][NB][4];
#pragma unroll
                for (int st = 0; st < kSteps; ++st) {
                    // the scale words of keys g and g + 8: K's (D = 64: K's and V's)
                    const uint32_t u0 = lds32(rd + at_s + 16 * st * L::kScaleRow), u1 = lds32(rd + at_s + (16 * st + 8) * L::kScaleRow);
                    float s0[2], s1[2], z0[2], z1[2];    // scales; zeros, as the codes are, times 2^-24
                    halves<BF16>(u0 & kScaleBits, s0[0], s0[1]);
                    halves<BF16>(u1 & kScaleBits, s1[0], s1[1]);
                    halves<false>(u0 & kM0, z0[0], z0[1]);
                    halves<false>(u1 & kM0, z1[0], z1[1]);
#pragma unroll
                    for (int gr = 0; gr < kGroups; ++gr) {
                        const uint2 a = lds64(rd + at_k[gr] + 16 * st * L::kRow), b = lds64(rd + at_k[gr] + (16 * st + 8) * L::kRow);
                        const uint32_t aw[2] = {a.x, a.y}, bw[2] = {b.x, b.y};
                        float acc[NB][4];
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                acc[nb][e] = 0.f;
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            const uint32_t a8 = aw[w] >> 8, b8 = bw[w] >> 8;
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb) {
                                mma_f16_16816(acc[nb], aw[w] & kM0, bw[w] & kM0, a8 & kM0, b8 & kM0, qf[nb][gr][2 * w][0],
                                              qf[nb][gr][2 * w][1]);
                                mma_f16_16816(acc[nb], aw[w] & kM1, bw[w] & kM1, a8 & kM1, b8 & kM1, qf[nb][gr][2 * w + 1][0],
                                              qf[nb][gr][2 * w + 1][1]);
                            }
                        }
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float x = fmaf(e < 2 ? z0[gr] : z1[gr], qs[nb][gr][e & 1], acc[nb][e]);
                                s[st][nb][e] = gr == 0 ? x * (e < 2 ? s0[gr] : s1[gr]) : fmaf(x, e < 2 ? s0[gr] : s1[gr], s[st][nb][e]);
                            }
                    }
                }
                if ((kb < all_lo && kb + kWarpKeys > p.sinks) || kb + kWarpKeys - 1 > all_hi) {
#pragma unroll
                    for (int st = 0; st < kSteps; ++st)
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int place = kb + 16 * st + key_row(g) + (e < 2 ? 0 : 8);
                                if ((place < see[nb][e & 1].x && place >= p.sinks) || place > see[nb][e & 1].y)
                                    s[st][nb][e] = -INFINITY;
                            }
                }
                // a new maximum of some row?
                float most[NB][2];
                bool up = false;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        most[nb][e] = fmaxf(s[0][nb][e], s[0][nb][2 + e]);
#pragma unroll
                        for (int st = 1; st < kSteps; ++st)
                            most[nb][e] = fmaxf(most[nb][e], fmaxf(s[st][nb][e], s[st][nb][2 + e]));
                        up |= most[nb][e] > limit[nb][e];
                    }
                if (__any_sync(0xffffffffu, up)) {
                    // exponents of the V scales (of a step's keys g and g + 8): a row's first f follows from them
                    // and the scores (by the pass below, like later ones, 64 sequences took 53.4 us)
                    float ea[kSteps][2][kGroups];
#pragma unroll
                    for (int st = 0; st < kSteps; ++st)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float a[2];
                            halves<BF16>(lds32(rd + at_s + (16 * st + 8 * k) * L::kScaleRow + (kGroups == 2 ? 4 : 0)) & kScaleBits, a[0], a[1]);
#pragma unroll
                            for (int gr = 0; gr < kGroups; ++gr)
                                ea[st][k][gr] = static_cast<float>(static_cast<int>(__float_as_uint(a[kGroups == 2 ? gr : 1]) >> 23) - 127);
                        }
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float x = most[nb][e], c[kGroups];
#pragma unroll
                            for (int gr = 0; gr < kGroups; ++gr) {
                                c[gr] = -INFINITY;
#pragma unroll
                                for (int st = 0; st < kSteps; ++st)
                                    c[gr] = fmaxf(c[gr], fmaxf(fmaf(s[st][nb][e], rowf[nb][e], ea[st][0][gr]), fmaf(s[st][nb][2 + e], rowf[nb][e], ea[st][1][gr])));
                            }
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) {
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
#pragma unroll
                                for (int gr = 0; gr < kGroups; ++gr)
                                    c[gr] = fmaxf(c[gr], __shfl_xor_sync(0xffffffffu, c[gr], d));
                            }
                            if (x > limit[nb][e]) {
                                x *= rowf[nb][e];
                                const bool none = limit[nb][e] == -INFINITY;
                                // the largest score itself, so that its weight is a power of two and its product with a
                                // scale exact.  The sum falls; f rises by whole powers of two, the output falls by the rest
                                const float by = none ? 0.f : fminf(fmaxf(x + minus[nb][e] - kShift, 0.f), 1024.f);
                                l[nb][e] *= ex2(-by);
                                minus[nb][e] = kShift - x;
                                limit[nb][e] = (x + kGrow) / rowf[nb][e];
#pragma unroll
                                for (int gr = 0; gr < kGroups; ++gr) {
                                    const int was = static_cast<int>(__float_as_uint(f[nb][gr][e]) >> 23);
                                    const int now = none ? 127 + 6 - static_cast<int>(fminf(fmaxf(c[gr] + minus[nb][e], 6 - 112.f), 120.f))
                                                         : min(was + static_cast<int>(by), kMostF);
                                    f[nb][gr][e] = __uint_as_float(static_cast<uint32_t>(now) << 23);
                                    if (!none)
                                        scale_output(o[nb][gr], oz[nb][gr], e, ex2(static_cast<float>(now - was) - by));
                                }
                            }
                        }
                }
                // weights; times their keys' V scales the right operand, turned over below
                uint32_t pf[kSteps][NB][kGroups][2];
                auto weighted = [&](bool first) {
                    uint32_t top = 0;
#pragma unroll
                    for (int st = 0; st < kSteps; ++st) {
                        float v0[2], v1[2];              // V scales of keys g and g + 8
                        halves<BF16>(lds32(rd + at_s + 16 * st * L::kScaleRow + (kGroups == 2 ? 4 : 0)) & kScaleBits, v0[0], v0[1]);
                        halves<BF16>(lds32(rd + at_s + (16 * st + 8) * L::kScaleRow + (kGroups == 2 ? 4 : 0)) & kScaleBits, v1[0], v1[1]);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            float(&w)[4] = s[st][nb];
                            if (first) {
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    w[e] = ex2(fmaf(w[e], rowf[nb][e & 1], minus[nb][e & 1]));
                                l[nb][0] += w[0] + w[2];
                                l[nb][1] += w[1] + w[3];
                            }
#pragma unroll
                            for (int gr = 0; gr < kGroups; ++gr) {
                                const float a = v0[kGroups == 2 ? gr : 1], b = v1[kGroups == 2 ? gr : 1];
                                pf[st][nb][gr][0] = pack16<false>(w[0] * f[nb][gr][0] * a, w[1] * f[nb][gr][1] * a);
                                pf[st][nb][gr][1] = pack16<false>(w[2] * f[nb][gr][0] * b, w[3] * f[nb][gr][1] * b);
                                top = max16x2(top, max16x2(pf[st][nb][gr][0], pf[st][nb][gr][1]));
                            }
                        }
                    }
                    return top;
                };
                // one that does not fit (an infinity): f comes down, and the output with it
                if (__any_sync(0xffffffffu, (weighted(true) + 0x04000400u) & 0x80008000u)) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int gr = 0; gr < kGroups; ++gr)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                // the largest, times 2^-16 (products of weights up to 2^15 and scales stay numbers)
                                float x = 0.f;
#pragma unroll
                                for (int st = 0; st < kSteps; ++st)
#pragma unroll
                                    for (int k = 0; k < 2; ++k) {
                                        float a[2];
                                        halves<BF16>(lds32(rd + at_s + (16 * st + 8 * k) * L::kScaleRow + (kGroups == 2 ? 4 : 0)) & kScaleBits,
                                                     a[0], a[1]);
                                        x = fmaxf(x, s[st][nb][2 * k + e] * 1.52587890625e-5f * a[kGroups == 2 ? gr : 1]);
                                    }
#pragma unroll
                                for (int d = 4; d < 32; d <<= 1)
                                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                                const int ex = static_cast<int>(__float_as_uint(x) >> 23), was = static_cast<int>(__float_as_uint(f[nb][gr][e]) >> 23);
                                if (ex + was >= 15 + 127 + 127 - 16) {   // 2^15 or more: to 2^7
                                    const int now = max(7 + 127 + 127 - 16 - ex, 1);
                                    f[nb][gr][e] = __uint_as_float(static_cast<uint32_t>(now) << 23);
                                    scale_output(o[nb][gr], oz[nb][gr], e, __uint_as_float(static_cast<uint32_t>(max(127 + now - was, 0)) << 23));
                                }
                            }
                    weighted(false);
                }
#pragma unroll
                for (int st = 0; st < kSteps; ++st) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int gr = 0; gr < kGroups; ++gr) {
                            pf[st][nb][gr][0] = transpose8(pf[st][nb][gr][0]);
                            pf[st][nb][gr][1] = transpose8(pf[st][nb][gr][1]);
                        }
                    // output: rows are d, columns query rows
                    uint32_t zw[4];                          // the V scale words of the keys 2 t, 2 t + 1, + 8
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        zw[i] = lds32(rd + at_z[i & 1] + (16 * st + 8 * (i >> 1)) * L::kScaleRow);
#pragma unroll
                    for (int gr = 0; gr < kGroups; ++gr) {
                        const uint32_t sel = kGroups == 2 && gr == 0 ? 0x5410u : 0x7632u;
                        const uint32_t z0 = __byte_perm(zw[0], zw[1], sel) & kM0, z1 = __byte_perm(zw[2], zw[3], sel) & kM0;
                        uint32_t v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[i] = lds32(rd + at_v[i & 1][gr] + (16 * st + 8 * (i >> 1)) * L::kRow);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {   // codes 0 .. 3, 4 .. 7 of the word
                            const uint32_t hs = half ? 0x7632u : 0x5410u;
                            const uint32_t a = __byte_perm(v[0], v[1], hs), b = __byte_perm(v[2], v[3], hs);
                            const uint32_t a8 = __byte_perm(a, 0u, 0x4341u), b8 = __byte_perm(b, 0u, 0x4341u);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb) {
                                mma_f16_16816(o[nb][gr][2 * half], a & kM0, a & kMB, b & kM0, b & kMB, pf[st][nb][gr][0], pf[st][nb][gr][1]);
                                mma_f16_16816(o[nb][gr][2 * half + 1], a8 & kM0, a8, b8 & kM0, b8, pf[st][nb][gr][0], pf[st][nb][gr][1]);
                            }
                        }
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
                            mma_f16_16816(oz[nb][gr], z0, 0u, z1, 0u, pf[st][nb][gr][0], pf[st][nb][gr][1]);
                    }
                }
            }
            __syncwarp();   // every lane has read the slot before it is filled again
            rd = next_stage(rd);
        }
        cp_async_wait_group<0>();
        // a row's sum and output count 2^(s - m) in bf16, 2^7 times that in fp16 (row_log_sum)
        constexpr float unshift = BF16 ? 1.f / 128 : 1.f;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                    l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], d);
                l[nb][e] *= unshift;
            }

        // the warps' maxima, sums and outputs meet in shared memory (over the rings)
        __syncthreads();
        float *wo = reinterpret_cast<float *>(smem);
        float *wml = reinterpret_cast<float *>(smem + L::kOffMl);
        constexpr float unit = 16777216.f * unshift;   // 2^24 for the codes
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = warp * kRows + 8 * nb + 2 * t + e;
#pragma unroll
                for (int gr = 0; gr < kGroups; ++gr) {
                    const float back = __uint_as_float((254u << 23) - __float_as_uint(f[nb][gr][e]));   // 1 / f
                    float *w = wo + row * L::kPitch + gr * kKv4Group + 8 * g;
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {    // values 2 i (of c), 2 i + 1 (of 16 c and the c before it)
                        v[2 * i] = (o[nb][gr][i][e] - oz[nb][gr][e]) * unit * back;
                        v[2 * i + 1] = fmaf(o[nb][gr][i][2 + e] - o[nb][gr][i][e], 0.0625f, -oz[nb][gr][e]) * unit * back;
                    }
                    *reinterpret_cast<float4 *>(w) = make_float4(v[0], v[1], v[2], v[3]);
                    *reinterpret_cast<float4 *>(w + 4) = make_float4(v[4], v[5], v[6], v[7]);
                }
                if (g == 0)
                    *reinterpret_cast<float2 *>(wml + row * 2) = make_float2(limit[nb][e] == -INFINITY ? -INFINITY : kShift - minus[nb][e], l[nb][e]);
            }
        __syncthreads();
        if (finish_rows<L, D, BF16, WARPS, kRows>(p, sg, smem))
            return;
        if (tid == 0 && is_last_part(sg))
            write_meta<kDecodeSetup>(p, sg, share.chunk);
        __syncthreads();   // the rings are free again
    }
}

template <int D, bool BF16, int WARPS, int NB>
cudaError_t decode_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&attr)[2], int grid, int cluster,
                          cudaStream_t stream)
{
    using L = Layout<D, WARPS, NB>;
    static SmemLimit limit;
    if (const cudaError_t e = ensure_smem_limit(limit, kv4_decode_kernel<D, BF16, WARPS, NB>, L::kClusterBytes, true);
        e != cudaSuccess)
        return e;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(32 * WARPS);
    cfg.dynamicSmemBytes = cluster > 1 ? L::kClusterBytes : L::kBytes;
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

template <int D, bool BF16, int WARPS, int NB>
cudaError_t launch_width(const Kv4AttnParams &p, int grid, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    if (const cudaError_t e = decode_config<D, BF16, WARPS, NB>(cfg, attr, grid, p.cluster, stream); e != cudaSuccess)
        return e;
    return cudaLaunchKernelEx(&cfg, kv4_decode_kernel<D, BF16, WARPS, NB>, p);
}

// Clusters of 2, 4 or 8 blocks that run at once on the current device: fewer than its
// blocks' number would give, since a cluster lies in one part of the device.
template <int D, bool BF16, int NB>
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
    if (decode_config<D, BF16, 8, NB>(cfg, attr, cluster, cluster, nullptr) != cudaSuccess)
        return 0;
    cfg.attrs = attr + 1;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kv4_decode_kernel<D, BF16, 8, NB>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    k.store(n + 1, std::memory_order_relaxed);
    return n;
}

template <int D, bool BF16>
cudaError_t launch_decode(const Kv4AttnParams &p, int grid, cudaStream_t stream)
{
    if (p.tile_rows == 8)
        return p.warps == 8 ? launch_width<D, BF16, 8, 1>(p, grid, stream) : launch_width<D, BF16, 4, 1>(p, grid, stream);
    return p.warps == 8 ? launch_width<D, BF16, 8, 2>(p, grid, stream) : launch_width<D, BF16, 4, 2>(p, grid, stream);
}

template <int D, bool BF16>
int clusters_of(int rows, int cluster)
{
    return rows == 8 ? active_clusters<D, BF16, 1>(cluster) : active_clusters<D, BF16, 2>(cluster);
}

}  // namespace

cudaError_t launch_kv4_decode(const Kv4AttnParams &p, int grid, cudaStream_t stream)
{
    const bool bf16 = p.kv.dtype == QMM_BF16;
    if (p.kv.head_dim == 128)
        return bf16 ? launch_decode<128, true>(p, grid, stream) : launch_decode<128, false>(p, grid, stream);
    return bf16 ? launch_decode<64, true>(p, grid, stream) : launch_decode<64, false>(p, grid, stream);
}

int kv4_decode_clusters(int head_dim, bool bf16, int rows, int cluster)
{
    if (head_dim == 128)
        return bf16 ? clusters_of<128, true>(rows, cluster) : clusters_of<128, false>(rows, cluster);
    return bf16 ? clusters_of<64, true>(rows, cluster) : clusters_of<64, false>(rows, cluster);
}

}  // namespace qmm
