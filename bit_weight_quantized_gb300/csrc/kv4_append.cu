// kv4_append.cu -- storing new keys and values in the 4-bit paged cache: keys (and the
// queries beside them) normed and rotated on the way, keys and values quantized.
//
//   y = x / sqrt(mean x^2 + eps) w               over a head, where there are weights
//   a' = a cos - b sin,  b' = b cos + a sin      for the rotated pairs, as in kv_append.cu
//   x = y' rounded to the type; for each 64 values of x:
//   lo = min(0, min x),  hi = max(0, max x),
//   s = (hi - lo) / 15 rounded up to 4 (bf16) or 7 (fp16) significant bits,
//   z = rint(-lo / s),  c = clamp(rint(x / s) + z, 0, 15)
//
// in fp32 with IEEE division and without fused multiply-adds, so that a plain computation
// step by step gives the same codes.  x / s is a tie exactly when the division says so: x and
// s have 11 and 7 bits at most, and a quotient that is no tie is further from one than
// fp32 rounds.
//
// Bound by memory, like kv_append.cu, whose layout this has: a block serves a token,
// thread i of a column of head_dim / 16 owns two 8-value chunks of a head.  The sums and the
// extremes of a head meet by shuffles within the column.
#include "kv4.cuh"

namespace qmm {

namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 2;                                // heads in flight per thread

// Smallest and largest of two pairs of 16-bit values; NaN where either is.
template <bool BF16>
__device__ __forceinline__ uint32_t min16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    if constexpr (BF16)
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

template <bool BF16>
__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    if constexpr (BF16)
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &w, float *x)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = lo16<BF16>(u[i]);
        x[2 * i + 1] = hi16<BF16>(u[i]);
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float *x)
{
    return make_uint4(pack16<BF16>(x[0], x[1]), pack16<BF16>(x[2], x[3]), pack16<BF16>(x[4], x[5]), pack16<BF16>(x[6], x[7]));
}

// (min, max) of a chunk with zero, one in each half of a word's place.
template <bool BF16>
__device__ __forceinline__ void extremes(const uint4 &w, uint32_t &lo, uint32_t &hi)
{
    uint32_t a = min16x2<BF16>(min16x2<BF16>(w.x, w.y), min16x2<BF16>(w.z, w.w));
    uint32_t b = max16x2<BF16>(max16x2<BF16>(w.x, w.y), max16x2<BF16>(w.z, w.w));
    lo = min16x2<BF16>(min16x2<BF16>(a, __byte_perm(a, a, 0x1032)), 0u);
    hi = max16x2<BF16>(max16x2<BF16>(b, __byte_perm(b, b, 0x1032)), 0u);
}

// A group's scale and zero from its extremes.
template <bool BF16>
struct Quant {
    float s, z;
    bool large;             // values near the type's largest: see code()
    uint32_t pattern;
    __device__ __forceinline__ Quant(float lo, float hi)
    {
        constexpr uint32_t kLow = BF16 ? (1u << 20) - 1 : (1u << 17) - 1;   // the bits that s does not have
        constexpr float kLarge = BF16 ? 1.5e38f : 32000.f;
        const float x = __fdiv_rn(__fsub_rn(hi * 0.5f, lo * 0.5f), 7.5f);   // (hi - lo may overflow)
        s = __uint_as_float((__float_as_uint(x) + kLow) & ~kLow);
        if (!BF16 && x < 6.103515625e-5f)                                   // below the normal numbers: steps of 2^-20
            s = ceilf(x * 1048576.f) * 9.5367431640625e-7f;
        z = s > 0.f ? fminf(rintf(__fdiv_rn(-lo, s)), 15.f) : 0.f;
        large = hi > kLarge || lo < -kLarge;
        pattern = (pack16<BF16>(s, 0.f) & 0xfff0u) | static_cast<uint32_t>(z);
        if (!(x < INFINITY)) {                                              // NaN or an infinity among the values
            s = z = 0.f;
            pattern = 0x7ff0u;                                              // (a NaN)
        }
        if (s == 0.f)
            z = 0.f;
    }
    __device__ __forceinline__ uint32_t code(float x) const
    {
        constexpr float kMost = BF16 ? 3.3895313892515355e38f : 65504.f;
        float c = s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(x, s)) + z, 0.f), 15.f) : 0.f;
        if (large) {                                                        // the value stays finite
            const float v = (c - z) * s;
            c += v > kMost ? -1.f : v < -kMost ? 1.f : 0.f;
        }
        return static_cast<uint32_t>(c);
    }
    // eight 16-bit values to a word of codes
    __device__ __forceinline__ uint32_t codes(const uint4 &w) const
    {
        float x[8];
        unpack8<BF16>(w, x);
        uint32_t d = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            d |= code(x[i]) << (4 * i);
        return d;
    }
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads)
kv4_append_kernel(const __grid_constant__ Kv4AppendParams p)
{
    constexpr int kItems = D / 16;                       // threads per head
    constexpr int kCols = kThreads / kItems;             // heads in flight
    constexpr int kGroups = D / kKv4Group;
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
            } else {
                a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
            }
    };
    fetch();
    uint4 wq0 = {}, wq1 = {}, wk0 = {}, wk1 = {};
    if (p.q_norm) {
        wq0 = *reinterpret_cast<const uint4 *>(p.q_norm + 8 * c0);
        wq1 = *reinterpret_cast<const uint4 *>(p.q_norm + 8 * c1);
    }
    if (p.k_norm) {
        wk0 = *reinterpret_cast<const uint4 *>(p.k_norm + 8 * c0);
        wk1 = *reinterpret_cast<const uint4 *>(p.k_norm + 8 * c1);
    }

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
    int page, slot;
    const bool place = find_slot(kv, p.by_page, seq, pos, p.status, page, slot);
    const long long at = page * kv.page_stride + slot * kv.slot_stride;
    const long long sat = scale_offset(p.sc, page, slot);

    // norm and rotation of a head's chunks, rounded to the type
    auto turned = [&](uint4 &xa, uint4 &xb, bool norm, const uint4 &w0, const uint4 &w1) {
        float x[8], y[8];
        unpack8<BF16>(xa, x);
        unpack8<BF16>(xb, y);
        if (norm) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                ss += x[i] * x[i] + y[i] * y[i];
#pragma unroll
            for (int d = 1; d < kItems; d <<= 1)
                ss += __shfl_xor_sync(0xffffffffu, ss, d);
            const float r = __frsqrt_rn(__fadd_rn(ss * (1.f / D), p.eps));
            float u[8], v[8];
            unpack8<BF16>(w0, u);
            unpack8<BF16>(w1, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = __fmul_rn(__fmul_rn(x[i], r), u[i]);
                y[i] = __fmul_rn(__fmul_rn(y[i], r), v[i]);
            }
        }
        if (turn) {
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float &e = i < 4 ? x[2 * i] : y[2 * i - 8], &o = i < 4 ? x[2 * i + 1] : y[2 * i - 7];
                    const float e0 = e, o0 = o;
                    e = __fsub_rn(__fmul_rn(e0, cs[i]), __fmul_rn(o0, sn[i]));
                    o = __fadd_rn(__fmul_rn(o0, cs[i]), __fmul_rn(e0, sn[i]));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x0 = x[i], y0 = y[i];
                    x[i] = __fsub_rn(__fmul_rn(x0, cs[i]), __fmul_rn(y0, sn[i]));
                    y[i] = __fadd_rn(__fmul_rn(y0, cs[i]), __fmul_rn(x0, sn[i]));
                }
            }
        }
        xa = pack8<BF16>(x);
        xb = pack8<BF16>(y);
    };
    // the whole warp goes through this together: the heads' columns exchange values
    const int last = (heads + kBatch * kCols - 1) / (kBatch * kCols);
    for (int round = 0; round < last; ++round) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int hu = h + u * kCols;
            const bool is_q = hu < hq, is_k = hu >= hq && hu < hq + hk;
            const bool norm = (is_q && p.q_norm) || (is_k && p.k_norm);
            // (the columns of a warp may hold queries, keys and values side by side)
            if (__any_sync(0xffffffffu, norm)) {
                uint4 xa = a[u], xb = b[u];
                turned(xa, xb, true, is_q ? wq0 : wk0, is_q ? wq1 : wk1);
                if (norm) {
                    a[u] = xa;
                    b[u] = xb;
                }
            }
            if (!norm && turn && (is_q || is_k))
                turned(a[u], b[u], false, wq0, wq1);
            if (is_q && hu < heads) {
                uint16_t *dst = p.q_out + (static_cast<long long>(t) * hq + hu) * D;
                *reinterpret_cast<uint4 *>(dst + 8 * c0) = a[u];
                *reinterpret_cast<uint4 *>(dst + 8 * c1) = b[u];
            }
            if (!__any_sync(0xffffffffu, hu >= hq && hu < heads))
                continue;
            // extremes of the groups, group g in half g of a word
            uint32_t lo0, hi0, lo1, hi1;
            extremes<BF16>(a[u], lo0, hi0);
            extremes<BF16>(b[u], lo1, hi1);
            uint32_t lo, hi;
            if constexpr (kGroups == 2) {
                const uint32_t m0 = c0 >> 3 ? 0xffff0000u : 0xffffu, m1 = c1 >> 3 ? 0xffff0000u : 0xffffu;
                lo = min16x2<BF16>(lo0 & m0, lo1 & m1);
                hi = max16x2<BF16>(hi0 & m0, hi1 & m1);
            } else {
                lo = min16x2<BF16>(lo0, lo1);
                hi = max16x2<BF16>(hi0, hi1);
            }
#pragma unroll
            for (int d = 1; d < kItems; d <<= 1) {
                lo = min16x2<BF16>(lo, __shfl_xor_sync(0xffffffffu, lo, d));
                hi = max16x2<BF16>(hi, __shfl_xor_sync(0xffffffffu, hi, d));
            }
            if (is_q || hu >= heads || !place)
                continue;
            const Quant<BF16> g0(lo16<BF16>(lo), lo16<BF16>(hi)), g1(hi16<BF16>(lo), hi16<BF16>(hi));
            const uint32_t w0 = (kGroups == 2 && c0 >> 3 ? g1 : g0).codes(a[u]);
            const uint32_t w1 = (kGroups == 2 && c1 >> 3 ? g1 : g0).codes(b[u]);
            const int head = is_k ? hu - hq : hu - hq - hk;
            uint8_t *dst = static_cast<uint8_t *>(is_k ? kv.k : kv.v) + at + head * kv.head_stride;
            *reinterpret_cast<uint32_t *>(dst + 4 * c0) = w0;
            *reinterpret_cast<uint32_t *>(dst + 4 * c1) = w1;
            if (item == 0) {
                uint16_t *sd = p.sc.base + sat + head * p.sc.head + (is_k ? 0 : kGroups);
                if constexpr (kGroups == 2)
                    *reinterpret_cast<uint32_t *>(sd) = g0.pattern | g1.pattern << 16;
                else
                    *sd = static_cast<uint16_t>(g0.pattern);
            }
        }
        h += kBatch * kCols;
        if (round + 1 < last)
            fetch();
    }
}

template <int D, bool BF16>
cudaError_t launch_append(const Kv4AppendParams &p, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.kv.tokens);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4_append_kernel<D, BF16>, p);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendParams &p, cudaStream_t stream)
{
    const bool bf16 = p.kv.dtype == QMM_BF16;
    if (p.kv.head_dim == 128)
        return bf16 ? launch_append<128, true>(p, stream) : launch_append<128, false>(p, stream);
    return bf16 ? launch_append<64, true>(p, stream) : launch_append<64, false>(p, stream);
}

}  // namespace qmm
