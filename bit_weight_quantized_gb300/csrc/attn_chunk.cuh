// attn_chunk.cuh -- attention over the paged cache for many query rows per key head
// (chunks of a prompt, whole prompts), on the 5th-generation tensor cores.
//
//   S = Q K^T,  P = 2^(S scale log2(e) - m),  O += P V,  out = O / sum P
//
// A work item is 256 rows ((token, query head) pairs of one key head, so that a
// key tile loaded once serves all query heads that share it) as two streams of 128
// rows (or somewhat fewer, where the query heads per key head do not divide 128: a
// stream holds whole tokens, so that one tensor copy per 64 values brings its queries);
// the keys go by in tiles of 128.  Both products run on tcgen05 with their accumulators
// in tensor memory: per stream S (128 x 128 fp32) and O (128 x D), all 512 columns at
// D = 128.  P takes S's place as 16-bit values and is the second
// product's left operand straight from tensor memory; V is its right operand as it
// lies in the cache ([key][d], the "MN-major" form), so nothing is transposed.  An
// item of one stream's rows gives both streams the same rows and every other tile;
// stream 0 adds up the two at the end, straight from tensor memory.  The next item's
// queries are loaded, and its first scores computed, as soon as the last scores of this
// one are there.
//
// Roles.  Warps 0-3 and 4-7 are the softmax of streams 0 and 1, one thread per row:
// no exchange between lanes.  Warp 8 issues the products, one stream after the
// other, so that one's products run under the other's softmax.  (A warp for each
// stream let the two fall into step, with both softmaxes and then both products at
// once: 240 instead of 190 us for 4096 x 4096 x 32 heads of 128.)  Warp 9 finds the
// segments of the block's share ahead of the others and brings their queries.  Warps 10
// and 11 bring K and V tiles into a ring each: where the page size is a multiple of 8 by
// tensor copies, one per page or part of a page that lies in the tile; else by
// 16-byte asynchronous copies, which take any page size.  V rows that nobody sees
// (past kv_len, before the window) are made zero, since 0 x NaN would spoil the
// product.  Plain copies kept the loading warps busy for 6000 cycles a tile pair,
// three times the products' time; plain copies of 256 query rows 3000 of all eight
// softmax warps' time, or 14000 of one warp's.
//
// Code that runs once per item costs some 6 cycles an instruction, since it has to be
// fetched: masks and outputs go through loops of 32 columns (straight code for the mask
// of a tile took 2500 cycles, the loop 1100 at most).
//
// The running maximum is replaced only when it grows by more than 2^8: the output
// accumulator in tensor memory is then read, scaled and written back by its
// stream's own threads, a few times per item.  S's arrival says that the product
// before it into O is complete, so that needs no signal of its own (D = 64, where the
// next S is computed under it: pv_done).
//
// The 4-bit cache (Q4) has the same tiles out of codes: two warps copy codes and scale
// patterns as they lie in the cache into a ring, four turn them into values (exact in the
// type) in the K and V rings.  Four warps that fetched codes by plain loads took 4500 cycles for
// a pair of tiles, half of it for ten loads in a queue behind the softmax's instructions (512
// tokens over 16384 keys 126 us, now 107; 97 without the conversions, as over the 16-bit
// cache).  Not kept: eight converting warps (120; fewer registers for the softmax),
// exponentials by a polynomial on the FMA pipe for every fourth weight (140).
//
// Bound by the tensor cores at D = 128 (a causal prompt of 8192 tokens x 64 heads: 1655
// TFLOP/s, 88% of the measured bf16 burst rate, until the power limit brings it to 1500;
// products and signals alone, the softmax left out, 1687 for 4096 x 4096 x 32), by the
// issuing warp and the softmax at D = 64 (4096 x 4096 x 32 heads: 132 us, 1041).
#pragma once

#include "gemm.cuh"
#include "kv4.cuh"

namespace qmm {

namespace {

constexpr int kSoftWarps = 4;                       // per stream
constexpr int kIssueWarp = 2 * kSoftWarps;
constexpr int kWalkWarp = kIssueWarp + 1, kLoadWarpV = kIssueWarp + 3;   // (K: the one between)
constexpr int kSegs = 4;                            // segments found ahead
constexpr float kChunkGrow = 8.f;
constexpr int kHalf = kChunkKeys / 2;               // the weights are handed over by halves of a tile
// The 16-bit cache's form and the 4-bit cache's (Q4).  Registers per thread after the split:
// 256 x 200 + 128 x 104 = 384 x 168, what the launch gives; Q4 256 x 192 + 256 x 64 = 512 x 128.
template <int D, bool Q4>
struct ChunkForm {
    using Params = AttnParams;
    static constexpr int kThreads = 384, kSoftRegs = 200, kOtherRegs = 104;
    static constexpr int kFillers = 1;                  // arrivals that make a K or V tile full
    static constexpr int kReaders = 2 * kSoftWarps + 3; // warps that go through the segments
    static constexpr int kKRing = D == 64 ? 5 : 3, kVRing = D == 64 ? 5 : 2, kRaw = 0;   // tiles of each ring
    static_assert(256 * kSoftRegs + 128 * kOtherRegs == kThreads * 168, "register split");
};
template <int D>
struct ChunkForm<D, true> {
    using Params = Kv4AttnParams;
    static constexpr int kThreads = 512, kSoftRegs = 192, kOtherRegs = 64;
    static constexpr int kFillers = 4;
    static constexpr int kReaders = 2 * kSoftWarps + 7;
    static constexpr int kKRing = D == 64 ? 5 : 2, kVRing = D == 64 ? 5 : 2, kRaw = D == 64 ? 6 : 3;
    static_assert(256 * kSoftRegs + 256 * kOtherRegs == kThreads * 128, "register split");
};
constexpr int kRawWarp = 10, kDequantWarp = 12;         // Q4: the first of the two and of the four

template <int D, bool Q4>
struct ChunkLayout {
    using Form = ChunkForm<D, Q4>;
    static constexpr int kTile = 128 * D * 2;       // 128 rows of D values: D / 64 halves of [128][64]
    static constexpr int kOffQ = 0;                 // two streams
    static constexpr int kKRing = Form::kKRing, kVRing = Form::kVRing;
    static constexpr int kOffK = 2 * kTile;
    static constexpr int kOffV = kOffK + kKRing * kTile;
    // Q4: codes of a K or V tile as they lie in the cache, and a word of patterns per key
    static constexpr int kRawCodes = 128 * D / 2, kRawStage = kRawCodes + 128 * 4;
    static constexpr int kOffRaw = kOffV + kVRing * kTile;
    static constexpr int kOffBar = kOffRaw + Form::kRaw * kRawStage;
    // full / empty of both rings, patch, per stream q_full, q_empty, s_full, p_full (two halves) and
    // pv_done, o_full, x_full, x_done, drain, full / empty of the segments and of the raw ring
    static constexpr int kNumBars = 2 * (kKRing + kVRing) + 18 + 2 * kSegs + 2 * Form::kRaw;
    static constexpr int kOffTmem = kOffBar + 8 * kNumBars;
    static constexpr int kOffShare = kOffTmem + 16;
    static constexpr int kOffRed = kOffShare + sizeof(Share);
    static constexpr int kOffSeg = kOffRed + 8 * 16;
    static constexpr int kOffX = (kOffSeg + static_cast<int>(sizeof(Segment)) * kSegs + 7) / 8 * 8;   // stream 1's maxima and sums
    static constexpr int kBytes = kOffX + 128 * 8;
    static_assert(kOffShare % 8 == 0 && sizeof(Share) % 8 == 0, "alignment");
    static_assert(kBytes <= 227 * 1024, "shared memory per block");
};

// Tensor-memory columns of stream s: S, half h of P, and O.  At D = 64 there is room for
// P beside S, so that the next scores are computed while the weights still are.
template <int D>
constexpr bool kBeside = D == 64;
__device__ __forceinline__ uint32_t s_col(int s) { return static_cast<uint32_t>(s) * 128u; }
template <int D>
__device__ __forceinline__ uint32_t p_col(int s, int h)
{
    return (kBeside<D> ? 384u + static_cast<uint32_t>(s) * 64u : s_col(s)) + static_cast<uint32_t>(h) * 32u;
}
template <int D>
__device__ __forceinline__ uint32_t o_col(int s) { return 256u + static_cast<uint32_t>(s * D); }

// Query tiles lie as halves of 64 values, rows of 128 bytes, chunks of 16 bytes permuted
// by the row (the 128-byte swizzle).

// Byte of chunk c of row r in a K or V tile: groups of 8 keys, each [D / 64 halves][8 keys][64
// values], so that one tensor copy brings both halves of a page's keys.
template <int D>
__device__ __forceinline__ uint32_t kv_addr(int r, int c)
{
    return static_cast<uint32_t>((r >> 3) * (D * 16) + (c >> 3) * 1024 + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// Byte of 16-byte piece c of key r in a tile of codes (Q4).
template <int D>
__device__ __forceinline__ uint32_t raw_addr(int r, int c)
{
    return static_cast<uint32_t>(r * (D / 2) + ((D == 128 ? c ^ (r >> 1 & 3) : c ^ (r >> 2 & 1)) << 4));
}

// Operand descriptor with the 128-byte swizzle.  `stride`: bytes between groups of 8
// rows (keys); `lead`: bytes between blocks of 64 values along the N index where the
// tile is read along d (MN-major), unused otherwise.
__device__ __forceinline__ uint64_t swizzled_desc(uint32_t saddr, uint32_t lead, uint32_t stride)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFF);
    d |= static_cast<uint64_t>((lead >> 4) & 0x3FFF) << 16;
    d |= static_cast<uint64_t>((stride >> 4) & 0x3FFF) << 32;
    d |= static_cast<uint64_t>(1) << 46;                            // descriptor version (tcgen05)
    d |= static_cast<uint64_t>(2) << 61;                            // 128-byte swizzle
    return d;
}

// D[tmem] (+)= A[tmem] * B[smem desc], kind::f16, one CTA
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// True in one lane of the (converged) warp, the same one every time.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(p));
    return p != 0;
}

// 32 tensor-memory columns of this thread's lane, without waiting
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// The same, and the largest of the 32 as fp32 values (NaN left out), without waiting
__device__ __forceinline__ void tmem_ld32_max_start(uint32_t taddr, uint32_t *r, float &most)
{
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=f"(most)
        : "r"(taddr));
}

// 5-D tiled load of a box into shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void *tmap, uint64_t *bar, int c3, int c4)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %3, %3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(0), "r"(c3), "r"(c4)
        : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, uint64_t *bar, int c0, int c1, int c2)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Ties 32 loaded registers to a point after the wait, so that no use moves above it.
__device__ __forceinline__ void pin32(uint32_t *r)
{
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
    asm volatile(""
                 : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31]));
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
        "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
        "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 values in one 64-bit register: the FMA pipe takes both in one
// instruction, which halves the softmax's issue slots there.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}

__device__ __forceinline__ void unpair(uint64_t v, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Chunks (16 bytes) of a group of four lanes, lane q's own four in a: afterwards lane q
// holds chunk q of the group's lanes in order.
__device__ __forceinline__ void transpose4(uint32_t (&a)[4][4], int lane)
{
#pragma unroll
    for (int d = 1; d <= 2; d <<= 1) {
        const bool odd = lane & d;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (c & d)
                continue;
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? a[c][f] : a[c + d][f], d);
                if (odd)
                    a[c][f] = got;
                else
                    a[c + d][f] = got;
            }
        }
    }
}

// An item of at most one stream's rows is shared by both streams, tile by tile.
__device__ __forceinline__ bool in_two(const Segment &s, int stream_rows) { return s.r.rows <= stream_rows && s.units > 1; }

template <int D, bool BF16, bool Q4>
__global__ void __launch_bounds__(ChunkForm<D, Q4>::kThreads, 1)
attn_chunk_kernel(const __grid_constant__ typename ChunkForm<D, Q4>::Params p)
{
    using L = ChunkLayout<D, Q4>;
    using Form = ChunkForm<D, Q4>;
    constexpr int kChunks = D / 8;                     // 16-byte chunks per row
    constexpr int kRowsPerCopy = 32 / kChunks;
    constexpr float kShift = BF16 ? 0.f : 7.f;
    // the operand tiles' swizzle needs 1024-byte alignment, which the start of a
    // block's shared memory has (there is no static part); checked below
    extern __shared__ __align__(1024) uint8_t smem[];
    Share &share = *reinterpret_cast<Share *>(smem + L::kOffShare);
    long long *red = reinterpret_cast<long long *>(smem + L::kOffRed);
    uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + L::kOffBar), *k_empty = k_full + L::kKRing;
    uint64_t *v_full = k_empty + L::kKRing, *v_empty = v_full + L::kVRing, *patch = v_empty + L::kVRing;
    uint64_t *q_full = patch + 1, *q_empty = q_full + 2, *s_full = q_empty + 2, *p_full = s_full + 2, *o_full = p_full + 4;
    uint64_t *x_full = o_full + 2, *x_done = x_full + 1, *drain = x_done + 1;
    uint64_t *pv_done = drain + 1, *seg_full = pv_done + 2, *seg_empty = seg_full + kSegs;
    [[maybe_unused]] uint64_t *raw_full = seg_empty + kSegs, *raw_empty = raw_full + Form::kRaw;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kOffTmem);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (smem_u32(smem) & 1023u) {
        if (threadIdx.x == 0)
            record_error(p.status, QMM_ERR_ALIGN);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < L::kKRing; ++i) {
            mbar_init(&k_full[i], Form::kFillers);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < L::kVRing; ++i) {
            mbar_init(&v_full[i], Form::kFillers);
            mbar_init(&v_empty[i], 1);
        }
        mbar_init(patch, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], 1);
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[2 * s], kSoftWarps);
            mbar_init(&p_full[2 * s + 1], kSoftWarps);
            mbar_init(&o_full[s], 1);
            mbar_init(&pv_done[s], 1);
        }
        mbar_init(x_full, kSoftWarps);
        mbar_init(x_done, kSoftWarps);
        mbar_init(drain, 1);
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(&seg_full[i], 1);
            mbar_init(&seg_empty[i], Form::kReaders);   // softmax, issue and loading warps
        }
        for (int i = 0; i < Form::kRaw; ++i) {
            mbar_init(&raw_full[i], 64);                    // the threads that copy
            mbar_init(&raw_empty[i], 4);
        }
        fence_barrier_init();
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    if (warp == kIssueWarp)
        tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!p.whole && threadIdx.x == 0)
        p.meta[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
    find_share<kChunkKeys, kChunkSetup, Form::kThreads, Q4>(p, red, &share);

    const int srows = chunk_stream_rows(p.group);   // a stream's rows
    bool ok = true;
    // Warp 9 walks the share and puts the segments, numbered, into a ring of kSegs; one
    // of no units ends them.  Every other warp goes through all of them.
    Segment *segs = reinterpret_cast<Segment *>(smem + L::kOffSeg);
    auto segment = [&](int n) -> const Segment & {
        if (ok)
            ok = __all_sync(0xffffffffu, mbar_wait(&seg_full[n % kSegs], n / kSegs & 1, p.status));
        return segs[n % kSegs];
    };
    auto leave = [&](int n) {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&seg_empty[n % kSegs]);
    };

    if (warp < kIssueWarp) {
        // ================= softmax of stream s: one row per thread =================
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Form::kSoftRegs));
        const int s = warp / kSoftWarps, quarter = warp % kSoftWarps;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t ts = tmem + lanes + s_col(s), to = tmem + lanes + o_col<D>(s);
        const uint32_t tp = tmem + lanes + p_col<D>(s, 0);
        float2 *x_ml = reinterpret_cast<float2 *>(smem + L::kOffX);
        uint32_t ph = 0;         // parity of the next S
        uint32_t oph = 0;        // parity of the next O
        uint32_t dph = 1;        // parity of the last tile's products into O (none at first)
        uint32_t xph = 0;        // parity of the next exchange between the streams
        for (int n = 0;; ++n) {
            const Segment &sg = segment(n);
            const RowTile r = sg.r;
            const int h = sg.h, units = sg.units, kb0 = (r.unit0 + sg.off) * kChunkKeys, slot = part_slot(sg);
            const bool two = in_two(sg, srows), whole = is_whole(sg);
            if (!ok || units == 0)
                break;
            if (threadIdx.x == 0 && is_last_part(sg))
                write_meta<kChunkSetup>(p, sg, share.chunk);
            leave(n);
            if (r.rows <= srows * s && !two)
                continue;                   // no rows of this stream's
            const int row = quarter * 32 + lane, trow = (two ? 0 : srows * s) + row;   // row in the stream, in the item
            const bool mine = row < srows && trow < r.rows;   // (the others hold anything)
            const int rr = r.row0 + trow;
            const int2 see = Q4 ? row_places(p, r, rr) : row_keys(p, r, rr);   // (Q4: kb and these are places)
            float mref = -INFINITY, l = 0.f;
            const uint64_t scale2 = pair(__float_as_uint(p.scale_log2), __float_as_uint(p.scale_log2));
            const int j0 = two ? s : 0, step = two ? 2 : 1;
            // keys that every row of the warp sees: halves inside need no mask
            int all_lo = mine ? see.x : 0, all_hi = mine ? see.y : 0x7fffffff;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, d));
                all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, d));
            }
            for (int j = j0; j < units; j += step) {
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(&s_full[s], ph, p.status))))
                    break;
                ph ^= 1u;
                tc_fence_after();
                const int kb = kb0 + j * kChunkKeys;
                // (Q4: the first tokens, before the window, are seen by all)
                auto all_see = [&](int k, int n) {
                    return (k >= all_lo || (Q4 && k + n <= p.sinks)) && k + n - 1 <= all_hi;
                };
                if (!all_see(kb, kChunkKeys)) {
                    // Keys that the row does not see get the score -infinity.  In place and
                    // in a loop: straight code for 128 columns, which few tiles run, took
                    // 2500 cycles of instruction fetches.
#pragma unroll 1
                    for (int c = 0; c < kChunkKeys; c += 32) {
                        if (all_see(kb + c, 32))
                            continue;
                        const int lo = see.x - kb - c, hi = see.y - kb - c;     // the columns this row sees
                        uint32_t above = lo <= 0 ? ~0u : lo > 31 ? 0u : ~0u << lo;
                        if constexpr (Q4) {
                            const int first = p.sinks - kb - c;
                            above |= first >= 32 ? ~0u : first <= 0 ? 0u : (1u << first) - 1u;
                        }
                        const uint32_t bits = (hi >= 31 ? ~0u : hi < 0 ? 0u : (2u << hi) - 1u) & above;
                        uint32_t x[32];
                        tmem_ld32_start(ts + c, x);
                        tmem_ld_wait();
                        pin32(x);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(bits >> e & 1u))
                                x[e] = 0xff800000u;
                        tmem_st32(ts + c, x);
                    }
                    tmem_st_wait();
                }
                uint32_t v[kChunkKeys];
                float mx[kChunkKeys / 32];
#pragma unroll
                for (int c = 0; c < kChunkKeys; c += 32)
                    tmem_ld32_max_start(ts + c, v + c, mx[c / 32]);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < kChunkKeys; c += 32) {
                    pin32(v + c);
                    asm volatile("" : "+f"(mx[c / 32]));
                }
                const float m = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * p.scale_log2;
                bool done = !kBeside<D>;     // whether the last tile's products are known to be complete
                auto pv_complete = [&]() {
                    if (!done)
                        ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[s], dph, p.status));
                    done = true;
                    tc_fence_after();
                };
                const bool up = m > mref + kChunkGrow;
                if (__any_sync(0xffffffffu, up)) {
                    const float a = up ? ex2(mref - m) : 1.f;
                    mref = up ? m : mref;
                    l *= a;
                    if (j > j0) {
                        pv_complete();
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32];
                            tmem_ld32_start(to + c, o);
                            tmem_ld_wait();
                            pin32(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                            tmem_st32(to + c, o);
                        }
                    }
                }
                const float neg = kShift - (mref == -INFINITY ? 0.f : mref);
                const uint64_t neg2 = pair(__float_as_uint(neg), __float_as_uint(neg));
                // weights, rounded to 16 bits for the second product; the first half of them
                // is handed over while the second is computed.  At D = 128 the scores are
                // read again, which lets their registers go (four sequences of up to 1000
                // tokens 46.7 us against 47.6); at D = 64 the softmax is on every tile's path
                // and the reads would lengthen it (143 against 131 for 4096 x 4096 x 32).
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int c = 0; c < kChunkKeys / 32; ++c) {
                    uint32_t w[16];
                    uint32_t *x = v + 32 * c;
                    if constexpr (!kBeside<D>) {
                        tmem_ld32_start(ts + 32 * c, x);
                        tmem_ld_wait();
                        pin32(x);
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float p0, p1;
                        unpair(fma2(pair(x[2 * e], x[2 * e + 1]), scale2, neg2), p0, p1);
                        p0 = ex2(p0);
                        p1 = ex2(p1);
                        sum[e & 1] = add2(sum[e & 1], pair(__float_as_uint(p0), __float_as_uint(p1)));
                        w[e] = pack16<BF16>(p0, p1);
                    }
                    if (kBeside<D> && c == 2)    // (its place may still be read)
                        pv_complete();
                    tmem_st16(tp + 16 * c, w);
                    if (c & 1) {
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(&p_full[2 * s + (c >> 1)]);
                    }
                }
                float s0, s1;
                unpair(add2(sum[0], sum[1]), s0, s1);
                l += s0 + s1;
                dph ^= 1u;
                if (!ok)
                    break;
            }
            if (ok)
                ok = __all_sync(0xffffffffu, mbar_wait(&o_full[s], oph, p.status));
            oph ^= 1u;
            if (!ok)
                break;
            tc_fence_after();
            // an item shared by both streams: stream 1 leaves its maximum and sum in
            // shared memory, stream 0 (same rows, same lanes) adds both up
            float w0 = 1.f, w1 = 0.f;
            if (two) {
                if (s == 1) {
                    x_ml[row] = make_float2(mref, l);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(x_full);
                    ok = __all_sync(0xffffffffu, mbar_wait(x_done, xph, p.status));
                    xph ^= 1u;
                    if (!ok)
                        break;
                    tc_fence_after();
                    continue;
                }
                ok = __all_sync(0xffffffffu, mbar_wait(x_full, xph, p.status));
                xph ^= 1u;
                if (!ok)
                    break;
                tc_fence_after();
                const float m1 = x_ml[row].x, l1 = x_ml[row].y;
                const float m = fmaxf(mref, m1), base = m == -INFINITY ? 0.f : m;
                w0 = ex2(mref - base);
                w1 = ex2(m1 - base);
                mref = m;
                l = w0 * l + w1 * l1;
            }
            // rows to memory: the item's output, or this block's part of it
            const float inv = row_inverse(l);
            float *part = p.part_o + static_cast<long long>(slot) * (kChunkRows * D) + 4 * trow;
            const int tok = p.by_group(rr), sub = lane & 3;
            // this row's place in the output, and those of the group of four lanes
            const long long place = mine ?
                (static_cast<long long>(r.t0 + tok) * p.q_heads + h * p.group + rr - tok * p.group) * D : -1;
            long long to_row[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                to_row[i] = __shfl_sync(0xffffffffu, place, (lane & ~3) + i);
            // (a loop, for the sake of the instruction fetches: see above)
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32_start(to + c, o);
                tmem_ld_wait();
                pin32(o);
                if (two) {
                    uint32_t o1[32];
                    tmem_ld32_start(tmem + lanes + o_col<D>(1) + c, o1);
                    tmem_ld_wait();
                    pin32(o1);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = __float_as_uint(w0 * __uint_as_float(o[e]) + w1 * __uint_as_float(o1[e]));
                }
                if (whole) {
                    // four lanes exchange their rows' pieces, so that each row's 64 bytes
                    // are stored by lanes side by side
                    uint32_t w[4][4];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        w[e >> 2][e & 3] = pack16<BF16>(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                    transpose4(w, lane);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (to_row[i] >= 0)
                            *reinterpret_cast<uint4 *>(p.out + to_row[i] + c + 8 * sub) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
                } else if (mine) {
                    // parts lie [D / 4][rows][4], so that a warp's rows are consecutive
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<uint4 *>(part + (c / 4 + e) * (4 * kChunkRows)) =
                            make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
            }
            tc_fence_before();   // the accumulators are read; the next P says so to the issuing warp
            __syncwarp();
            if (two && lane == 0)
                mbar_arrive(x_done);
            if (mine) {
                if (!whole)
                    *reinterpret_cast<float2 *>(p.part_ml + (static_cast<long long>(slot) * kChunkRows + trow) * 2) =
                        make_float2(mref, l);
                else if (p.lse)
                    p.lse[place / D] = row_log_sum<BF16>(mref, l);
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Form::kOtherRegs));
        if (warp == kIssueWarp) {
            // ================= product issue =================
            // The whole warp runs this, one elected lane issues: with warp-uniform
            // control flow the operand descriptors stay in uniform registers.  (A single
            // lane's loop spent 70 to 170 cycles a product on moving them there; a
            // product takes 64.)  A timed-out wait only skips the later waits: the loops
            // run on, over data that nobody uses.
            const uint32_t id_qk = f16_idesc(BF16, 128, kChunkKeys);
            const uint32_t id_pv = f16_idesc(BF16, 128, D) | (1u << 16);   // B is MN-major
            const uint64_t q_desc = swizzled_desc(smem_u32(smem + L::kOffQ), 16, 1024);
            const uint64_t k_desc = swizzled_desc(smem_u32(smem + L::kOffK), 16, D * 16);
            const uint64_t v_desc = swizzled_desc(smem_u32(smem + L::kOffV), 1024, D * 16);
            unsigned tile0 = 0;          // key tiles of the segments before
            uint32_t qph = 0, pph = 0;   // parities of q_full and p_full, bit per stream
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                if (ok)
                    ok = mbar_wait(bar, parity, p.status);
                tc_fence_after();
            };
            // wait for K or V tile j of the segment and return its slot
            auto k_landed = [&](int j) -> int {
                const unsigned at = tile0 + static_cast<unsigned>(j), slot = at % L::kKRing;
                wait(&k_full[slot], at / L::kKRing & 1u);
                return static_cast<int>(slot);
            };
            auto v_landed = [&](int j) -> int {
                const unsigned at = tile0 + static_cast<unsigned>(j), slot = at % L::kVRing;
                wait(&v_full[slot], at / L::kVRing & 1u);
                return static_cast<int>(slot);
            };
            // S of stream s from query tile qt and the K tile in slot ks; the last readers
            // free them
            auto qk = [&](int s, int qt, int ks, bool last, bool last_q) {
                const uint64_t a = q_desc + static_cast<uint32_t>((qt * L::kTile) >> 4);
                const uint64_t b = k_desc + static_cast<uint32_t>((ks * L::kTile) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        tc_mma(tmem + s_col(s), a + (kk >> 2) * (128 * 128 / 16) + (kk & 3) * 2,
                               b + (kk >> 2) * (1024 / 16) + (kk & 3) * 2, id_qk, kk > 0 ? 1u : 0u);
                    tc_commit(&s_full[s]);
                    if (last)
                        tc_commit(&k_empty[ks]);
                    if (last_q)
                        tc_commit(&q_empty[qt]);
                }
                __syncwarp();
            };
            // O of stream s (+)= P V for half h of a tile, V in slot vs, when its weights have
            // come
            auto pv = [&](int s, int h, int vs, bool first, bool last) {
                wait(&p_full[2 * s + h], pph >> s & 1u);
                const uint64_t b = v_desc + static_cast<uint32_t>((vs * L::kTile + h * (L::kTile / 2)) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int e = 0; e < kHalf / 16; ++e)
                        tc_mma_ts(tmem + o_col<D>(s), tmem + p_col<D>(s, h) + 8 * e, b + e * (2 * D * 16 / 16), id_pv,
                                  h > 0 || e > 0 || !first ? 1u : 0u);
                    if (kBeside<D> && h == 1)
                        tc_commit(&pv_done[s]);
                    if (h == 1 && last)
                        tc_commit(&v_empty[vs]);
                }
                if (h == 1) {
                    __syncwarp();
                    pph ^= 1u << s;
                }
            };
            auto finish = [&](int s) {   // stream s's last product of the segment
                if (elect_one())
                    tc_commit(&o_full[s]);
                __syncwarp();
            };
            auto q_landed = [&](int s) {
                wait(&q_full[s], qph >> s & 1u);
                qph ^= 1u << s;
            };
            for (int n = 0;; ++n) {
                const Segment &sg = segment(n);
                const int ns = __shfl_sync(0xffffffffu, sg.r.rows > srows ? 2 : 1, 0);
                const int units = __shfl_sync(0xffffffffu, sg.units, 0);
                if (!ok || units == 0)
                    break;
                leave(n);
                // (the streams' loops are unrolled: with constant streams a product issues
                // in 50 cycles, with variable ones in 60, and this warp is on every tile's
                // path; with a segment's first scores inside them, under a condition, 512 over
                // 16384 keys took 98 us instead of 89)
                if (ns == 1) {
                    // one stream's rows: even tiles on stream 0, odd ones on stream 1
                    q_landed(0);
                    qk(0, 0, k_landed(0), true, units == 1);
                    if (units > 1)
                        qk(1, 0, k_landed(1), true, units == 2);
                    for (int j0 = 0; j0 < units; j0 += 2) {
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            const int j = j0 + s;
                            if (j < units) {
                                const int vs = v_landed(j);
                                pv(s, 0, vs, j0 == 0, true);
                                if (!kBeside<D>)
                                    pv(s, 1, vs, j0 == 0, true);
                                if (j + 2 < units)
                                    qk(s, 0, k_landed(j + 2), true, j + 3 == units);
                                if (kBeside<D>)
                                    pv(s, 1, vs, j0 == 0, true);
                                if (j + 2 >= units)
                                    finish(s);
                            }
                        }
                    }
                } else {
                    int ks = k_landed(0);
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        q_landed(s);
                        qk(s, s, ks, s == 1, units == 1);
                    }
                    for (int j = 0; j < units; ++j) {
                        const int vs = v_landed(j);
                        const bool more = j + 1 < units;
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            pv(s, 0, vs, j == 0, s == 1);
                            if (!kBeside<D>)
                                pv(s, 1, vs, j == 0, s == 1);
                            if (more) {
                                if (s == 0)
                                    ks = k_landed(j + 1);
                                qk(s, s, ks, s == 1, j + 2 == units);
                            }
                            if (kBeside<D>)
                                pv(s, 1, vs, j == 0, s == 1);
                            if (!more)
                                finish(s);
                        }
                    }
                }
                tile0 += static_cast<unsigned>(units);
            }
            // after a timeout nobody has waited for the products: wait here
            if (!__all_sync(0xffffffffu, ok)) {
                if (elect_one())
                    tc_commit(drain);
                __syncwarp();
                mbar_wait(drain, 0, p.status);
            }
            __syncwarp();
        } else if (warp == kWalkWarp) {
            // ================= segments and query rows =================
            if (lane == 0) {
                Walk<kChunkKeys, kChunkSetup, Q4> walk;
                walk.begin(share);
                prefetch_tmap(&p.tmq);
                int found = 0;           // segments found
                bool more = true;
                uint32_t uses[2] = {0, 0};   // of the query tiles
                const int toks = 128 / p.group;
                for (int n = 0;; ++n) {
                    for (; more && found < n + (n == 0 ? 1 : kSegs); ++found) {
                        Segment &x = segs[found % kSegs];
                        if (found >= kSegs && !mbar_wait(&seg_empty[found % kSegs], (found / kSegs - 1) & 1, p.status)) {
                            ok = false;
                            break;
                        }
                        more = walk.next(p, x);
                        if (!more)
                            x.units = 0;
                        mbar_arrive(&seg_full[found % kSegs]);
                    }
                    const Segment &sg = segs[n % kSegs];
                    if (!ok || sg.units == 0)
                        break;
                    // its rows, whole tokens, into the query tiles (past the item: of whatever
                    // comes next)
                    const int ns = sg.r.rows > srows ? 2 : 1, tok = sg.r.t0 + p.by_group(sg.r.row0);
                    for (int s = 0; s < ns && ok; ++s) {
                        if (uses[s] > 0 && !(ok = mbar_wait(&q_empty[s], (uses[s] - 1) & 1u, p.status)))
                            break;
                        ++uses[s];
                        mbar_arrive_expect_tx(&q_full[s], static_cast<uint32_t>(srows * D * 2));
#pragma unroll
                        for (int c = 0; c < D; c += 64)
                            tma_load_3d(smem_u32(smem + L::kOffQ + s * L::kTile + c * 256), &p.tmq, &q_full[s], c,
                                        sg.h * p.group, tok + s * toks);
                    }
                }
                // no copy may still be landing when the block exits, also after a timeout
                for (int s = 0; s < 2; ++s)
                    if (uses[s] > 0)
                        mbar_wait(&q_full[s], (uses[s] - 1) & 1u, p.status);
            }
            __syncwarp();
        } else if constexpr (Q4) {
            if (warp < kDequantWarp) {
                // ================= codes (warps 10 and 11) =================
                // Lane l of a warp copies keys l and l + 32 of its half of every tile as they lie in
                // the cache, K and V in turn, and their words of patterns (zeros for keys that
                // nobody sees).  Pages are looked up a tile ahead.  16-byte pieces are permuted by
                // the key, so that eight threads that read a piece of a key each meet no bank twice.
                constexpr int kVecs = D / 32;
                const int row0 = 64 * (warp - kRawWarp) + lane;
                unsigned stage = 0;            // stages so far
                for (int n = 0; ok; ++n) {
                    const Segment &sg = segment(n);
                    const RowTile r = sg.r;
                    const int h = sg.h, units = sg.units, off = sg.off;
                    if (!ok || units == 0)
                        break;
                    leave(n);
                    const uint16_t *sbase = p.sc.base + h * p.sc.head;
                    // key i of the lane in tile j, -1 where nobody sees it, and its page
                    auto key_of = [&](int j, int i) {
                        if (j >= units)
                            return -1;
                        const int place = (off + j) * kChunkKeys + row0 + 32 * i;
                        return place < r.hi ? place + (place < p.sinks ? 0 : r.lo) : -1;
                    };
                    auto look_up = [&](int key) {
                        return key >= 0 ? p.kv.block_table[static_cast<long long>(r.b) * p.kv.blocks + p.by_page(key)] : 0;
                    };
                    int page[2] = {look_up(key_of(0, 0)), look_up(key_of(0, 1))};
                    for (int j = 0; j < units && ok; ++j) {
                        long long at[2], sat[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int key = key_of(j, i);
                            at[i] = -1;
                            sat[i] = 0;
                            if (key >= 0) {
                                if (page[i] < 0 || page[i] >= p.kv.num_pages) {
                                    record_error(p.status, QMM_ERR_INDEX);
                                } else {
                                    const int slot = key - p.by_page(key) * p.kv.page_size;
                                    at[i] = page[i] * p.kv.page_stride + slot * p.kv.slot_stride + h * p.kv.head_stride;
                                    sat[i] = scale_offset(p.sc, page[i], slot);
                                }
                            }
                            page[i] = look_up(key_of(j + 1, i));
                        }
#pragma unroll 1
                        for (int kk = 0; kk < 2; ++kk, ++stage) {
                            const unsigned slot = stage % Form::kRaw;
                            if (stage >= Form::kRaw &&
                                !(ok = __all_sync(0xffffffffu, mbar_wait(&raw_empty[slot], (stage / Form::kRaw - 1) & 1u, p.status))))
                                break;
                            const uint8_t *base = static_cast<const uint8_t *>(kk ? p.kv.v : p.kv.k);
                            const uint32_t dst = smem_u32(smem + L::kOffRaw) + slot * L::kRawStage;
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int row = row0 + 32 * i;
                                const bool in = at[i] >= 0;
                                const uint8_t *src = in ? base + at[i] : base;
#pragma unroll
                                for (int v = 0; v < kVecs; ++v)
                                    cp_async16_or_zero(dst + raw_addr<D>(row, v), src + 16 * v, in);
                                cp_async_small<4>(dst + L::kRawCodes + 4 * row,
                                                  sbase + sat[i] + (D == 128 && kk ? 2 : 0), in);
                            }
                            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&raw_full[slot])) : "memory");
                        }
                    }
                }
                cp_async_wait_all();   // no copy may still be landing when the block exits
            } else {
                // ================= K and V tiles out of codes (warps 12 - 15) =================
                // Thread r turns key r of every tile into values; 16-byte stores that eight threads
                // side by side make meet no bank twice.
                constexpr int kGroups = D / kKv4Group, kVecs = D / 32;
                const int row = threadIdx.x - 32 * kDequantWarp;
                unsigned tile = 0;             // tiles of each ring so far
                for (int n = 0; ok; ++n) {
                    const int units = segment(n).units;
                    if (!ok || units == 0)
                        break;
                    leave(n);
                    for (int i = 0; i < 2 * units; ++i) {
                        const bool v = i & 1;
                        const unsigned stage = 2 * tile + (v ? 1u : 0u), rs = stage % Form::kRaw;
                        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&raw_full[rs], stage / Form::kRaw & 1u, p.status))))
                            break;
                        const uint8_t *raw = smem + L::kOffRaw + rs * L::kRawStage;
                        uint4 w[kVecs];
#pragma unroll
                        for (int c = 0; c < kVecs; ++c)
                            w[c] = *reinterpret_cast<const uint4 *>(raw + raw_addr<D>(row, c));
                        const uint32_t pats = *reinterpret_cast<const uint32_t *>(raw + L::kRawCodes + 4 * row);
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(&raw_empty[rs]);
                        const unsigned ring = v ? L::kVRing : L::kKRing;
                        const unsigned slot = v ? tile % L::kVRing : tile % L::kKRing, use = v ? tile / L::kVRing : tile / L::kKRing;
                        if (tile >= ring &&
                            !(ok = __all_sync(0xffffffffu, mbar_wait(v ? &v_empty[slot] : &k_empty[slot], (use - 1) & 1u, p.status))))
                            break;
                        uint8_t *dst = smem + (v ? L::kOffV : L::kOffK) + slot * L::kTile;
#pragma unroll
                        for (int gr = 0; gr < kGroups; ++gr) {
                            const GroupScale<BF16> sc((kGroups == 2 ? gr == 1 : v) ? pats >> 16 : pats & 0xffffu);
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const uint4 x = w[2 * gr + c];
                                const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    *reinterpret_cast<uint4 *>(dst + kv_addr<D>(row, 8 * gr + 4 * c + e)) = sc.values(u[e]);
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(v ? &v_full[slot] : &k_full[slot]);
                        tile += v ? 1 : 0;
                    }
                }
            }
        } else {
            // ================= K tiles (warp 10) and V tiles (warp 11) =================
            const bool is_v = warp == kLoadWarpV;
            const int slots = is_v ? L::kVRing : L::kKRing;
            uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
            uint8_t *ring = smem + (is_v ? L::kOffV : L::kOffK);
            const CUtensorMap *map = is_v ? &p.tmv : &p.tmk;
            const int sub = lane / kChunks, chunk = lane % kChunks;
            const int nbox = p.box > 0 ? kChunkKeys / p.box : 0;     // tensor copies per tile, at most 16
            const uint32_t box_bytes = static_cast<uint32_t>(p.box * D * 2);
            int slot = 0, issued = 0;
            uint32_t par = 1;             // parity of the ring's empty barriers (none to wait for at first)
            uint32_t patched = 0;         // parity of the patch barrier
            int unsaid = -1;              // slot of a plain-copied tile that is not announced yet
            auto announce = [&]() {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&full[unsaid]);
            };
            if (lane == 0 && p.box > 0)
                prefetch_tmap(map);
            for (int n = 0; ok; ++n) {
                const Segment &sg = segment(n);
                const RowTile r = sg.r;
                const int h = sg.h, units = sg.units, kb0 = (r.unit0 + sg.off) * kChunkKeys;
                if (!ok || units == 0)
                    break;
                leave(n);
                const uint16_t *base = static_cast<const uint16_t *>(is_v ? p.kv.v : p.kv.k) + h * p.kv.head_stride;
                // page and slot / 8 of box `lane` of tile j (slot -1: nobody sees any of its
                // keys).  Looked up one tile ahead, and not looked at before it is used: the
                // warp would wait for the table's entry here.
                auto find_box = [&](int j) -> int2 {
                    const int key = kb0 + j * kChunkKeys + lane * p.box;
                    if (lane >= nbox || j >= units || key >= r.hi || key + p.box <= r.lo)
                        return make_int2(0, -1);
                    const int blk = p.by_page(key);
                    return make_int2(p.kv.block_table[static_cast<long long>(r.b) * p.kv.blocks + blk],
                                     (key - blk * p.kv.page_size) >> 3);
                };
                int2 at = find_box(0);
                for (int j = 0; j < units; ++j) {
                    const int kb = kb0 + j * kChunkKeys;
                    const int2 here = at;
                    at = find_box(j + 1);
                    if (issued >= slots && !(ok = __all_sync(0xffffffffu, mbar_wait(&empty[slot], par, p.status))))
                        break;
                    uint8_t *tile = ring + slot * L::kTile;
                    if (nbox > 0) {
                        // V rows that nobody sees must be zero (0 x NaN): such a tile lands on
                        // the patch barrier, the warp clears the rows and then says that the slot
                        // is full
                        const bool clear = is_v && (kb < r.lo || kb + kChunkKeys > r.hi);
                        const bool page_ok = here.x >= 0 && here.x < p.kv.num_pages;
                        if (here.y >= 0 && !page_ok)
                            record_error(p.status, QMM_ERR_INDEX);
                        const uint32_t mine = __ballot_sync(0xffffffffu, here.y >= 0 && page_ok);
                        uint64_t *bar = clear ? patch : &full[slot];
                        if (elect_one())
                            mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(mine)) * box_bytes);
                        __syncwarp();
                        // box by box, warp-uniform: lanes that issue side by side take turns
                        // anyway, and at several times the cost
                        const int row = here.x * p.page_step + h;
                        for (int x = 0; x < nbox; ++x) {
                            const int c3 = __shfl_sync(0xffffffffu, here.y, x), c4 = __shfl_sync(0xffffffffu, row, x);
                            if ((mine >> x & 1u) && elect_one())
                                tma_load_5d(smem_u32(tile) + static_cast<uint32_t>(x) * box_bytes, map, bar, c3, c4);
                            __syncwarp();
                        }
                        if (clear) {
                            if (!(ok = __all_sync(0xffffffffu, mbar_wait(patch, patched, p.status))))
                                break;
                            patched ^= 1u;
                            for (int q = sub; q < kChunkKeys; q += kRowsPerCopy)
                                if (kb + q < r.lo || kb + q >= r.hi)
                                    *reinterpret_cast<uint4 *>(tile + kv_addr<D>(q, chunk)) = make_uint4(0u, 0u, 0u, 0u);
                            unsaid = slot;
                            announce();
                            unsaid = -1;
                        }
                    } else {
                        // plain copies, 32 keys at a time: the lane looks up the place of one
#pragma unroll 1
                        for (int e = 0; e < kChunkKeys; e += 32) {
                            const int key = kb + e + lane;
                            const long long place = key >= r.lo && key < r.hi ? key_offset(p.kv, p.by_page, r.b, key, p.status) : -1;
#pragma unroll 4
                            for (int c = 0; c < 32; c += kRowsPerCopy) {
                                const long long o = __shfl_sync(0xffffffffu, place, c + sub);
                                cp_async16_or_zero(smem_u32(tile + kv_addr<D>(e + c + sub, chunk)),
                                                   o >= 0 ? base + o + chunk * 8 : p.q, o >= 0);
                            }
                        }
                        cp_async_commit();
                        // the tile before this one has landed
                        cp_async_wait_group<1>();
                        if (unsaid >= 0)
                            announce();
                        unsaid = slot;
                    }
                    ++issued;
                    if (++slot == slots) {
                        slot = 0;
                        par ^= 1u;
                    }
                }
            }
            if (unsaid >= 0) {
                cp_async_wait_group<0>();
                announce();
            }
            // no copy may still be landing when the block exits, also after a timeout
            if (lane == 0)
                for (int i = max(0, issued - slots); i < issued; ++i)
                    if (!mbar_wait(&full[i % slots], (i / slots) & 1, p.status))
                        break;
            __syncwarp();
        }
    }

    // teardown: every role is done (or gave up); release tensor memory
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kIssueWarp)
        tmem_dealloc(tmem, 512);
}

template <int D, bool BF16, bool Q4>
cudaError_t launch_chunk(const typename ChunkForm<D, Q4>::Params &p, int grid, cudaStream_t stream)
{
    constexpr int smem = ChunkLayout<D, Q4>::kBytes;
    static SmemLimit limit;
    if (const cudaError_t e = ensure_smem_limit(limit, attn_chunk_kernel<D, BF16, Q4>, smem, true); e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(ChunkForm<D, Q4>::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_chunk_kernel<D, BF16, Q4>, p);
}

template <bool Q4>
cudaError_t launch_chunk_form(const typename ChunkForm<64, Q4>::Params &p, int grid, cudaStream_t stream)
{
    const bool bf16 = p.kv.dtype == QMM_BF16;
    if (p.kv.head_dim == 128)
        return bf16 ? launch_chunk<128, true, Q4>(p, grid, stream) : launch_chunk<128, false, Q4>(p, grid, stream);
    return bf16 ? launch_chunk<64, true, Q4>(p, grid, stream) : launch_chunk<64, false, Q4>(p, grid, stream);
}

}  // namespace

}  // namespace qmm
