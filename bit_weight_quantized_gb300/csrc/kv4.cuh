// kv4.cuh -- device helpers of the 4-bit paged cache kernels.
//
// 64 values of a head share a scale s and a zero z: code c, 0 .. 15, stands for (c - z) s.
// s has 4 significant bits in bf16 and 7 in fp16, so that (c - z) s is exact in the type, and
// the low four bits of its pattern hold z.  Codes lie two to a byte, the low half first.
#pragma once

#include "kv4.h"
#include "paged.cuh"

namespace qmm {

namespace {

template <bool BF16>
__device__ __forceinline__ float scale_of(uint32_t pattern)
{
    return BF16 ? __uint_as_float((pattern & 0xfff0u) << 16) : f16_bits_to_f32(static_cast<uint16_t>(pattern & 0xfff0u));
}

// Two 16-bit products and sums, exact for the numbers they are used on.
template <bool BF16>
__device__ __forceinline__ uint32_t sub16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    if constexpr (BF16)
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

template <bool BF16>
__device__ __forceinline__ uint32_t mul16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    if constexpr (BF16)
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// What a group's codes need to become values: base + z and s, each twice in a word.  A code
// in the low bits of the pattern of `base` (128 in bf16, 1024 in fp16) is base + c, from
// which base + z is subtracted exactly.
template <bool BF16>
struct GroupScale {
    static constexpr uint32_t kBase = BF16 ? 0x43004300u : 0x64006400u;
    uint32_t zero, scale;
    __device__ __forceinline__ explicit GroupScale(uint32_t pattern)
    {
        zero = kBase | (pattern & 15u) * 0x10001u;
        scale = (pattern & 0xfff0u) * 0x10001u;
    }
    // eight codes (a word) to values in order
    __device__ __forceinline__ uint4 values(uint32_t w) const
    {
        const uint32_t y = w >> 4;
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // byte i: codes 2 i (from w) and 2 i + 1 (from y)
            const uint32_t both = __byte_perm(w, y, 0x0400u + 0x0101u * i);
            v[i] = mul16x2<BF16>(sub16x2<BF16>((both & 0x000f000fu) | kBase, zero), scale);
        }
        return make_uint4(v[0], v[1], v[2], v[3]);
    }
};

// 8 or 4 bytes global -> shared (zeros where !ok)
template <int BYTES>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src, bool ok)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(ok ? BYTES : 0)
                 : "memory");
}

__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Element offset of the scales of (page, slot, head 0).
__device__ __forceinline__ long long scale_offset(const Kv4Scales &sc, int page, int slot)
{
    return page * sc.page + slot * sc.slot;
}

// Page and slot of key `key` of sequence b; false (recorded) for a page number out of range.
__device__ __forceinline__ bool find_slot(const qmm_paged_kv &kv, const FastDiv &by_page, int b, int key, int *status,
                                          int &page, int &slot)
{
    const int blk = by_page(key);
    slot = key - blk * kv.page_size;
    page = kv.block_table[static_cast<long long>(b) * kv.blocks + blk];
    if (page < 0 || page >= kv.num_pages) {
        record_error(status, QMM_ERR_INDEX);
        return false;
    }
    return true;
}

}  // namespace

}  // namespace qmm
