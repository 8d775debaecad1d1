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
// in fp32 with correctly rounded quotients and, in the rotation, without fused multiply-adds, so
// that a plain computation step by step gives the same codes where there are no norms (whose sum of
// squares has an order of its own, and whose root is rsqrtf's).  x / s is a tie exactly when the
// division says so: x and s have 11 and 7 bits at most, and a quotient that is no tie is
// further from one than fp32 rounds.
//
// Bound by memory, like kv_append.cu, whose layout this has, and nearly as much by
// instructions: a block serves a token, thread i of a column of head_dim / 16 owns two 8-value
// chunks of a head.  The sums and the extremes of a head meet by shuffles within the column.
// 8192 tokens of 80 heads of 128: 61.4 us with norms, 53.9 without (5.1 and 5.8 TB/s); with
// divisions and one loop over all heads 93.
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

// Two fp32 values in one 64-bit register: the FMA pipe takes both in one instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}

__device__ __forceinline__ float2 unpair(uint64_t v)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// Eight 16-bit values as four pairs.
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &w, uint64_t *x)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = pair(lo16<BF16>(u[i]), hi16<BF16>(u[i]));
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const uint64_t *x)
{
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpair(x[i]);
        u[i] = pack16<BF16>(f.x, f.y);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
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
        // (half of hi - lo, which may overflow, rounded up; an s times 7.5 is exact)
        const float d = __fsub_ru(hi * 0.5f, lo * 0.5f), x = __fmul_rz(d, 0x1.11111p-3f);   // 1 / 7.5 and x are cut off
        s = __uint_as_float((__float_as_uint(x) + kLow) & ~kLow);
        float next = __uint_as_float(__float_as_uint(s) + kLow + 1);
        if (!BF16 && x < 6.103515625e-5f) {                                 // below the normal numbers: steps of 2^-20
            s = ceilf(x * 1048576.f) * 9.5367431640625e-7f;
            next = s + 9.5367431640625e-7f;
        }
        s = s * 7.5f < d ? next : s;                                        // where the quotient lies just above the cut one
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
    // what the neighbouring thread worked out (the whole warp)
    __device__ __forceinline__ Quant swapped() const
    {
        Quant q = *this;
        q.s = __shfl_xor_sync(0xffffffffu, s, 1);
        q.z = __shfl_xor_sync(0xffffffffu, z, 1);
        q.pattern = __shfl_xor_sync(0xffffffffu, pattern, 1);
        q.large = __shfl_xor_sync(0xffffffffu, large, 1);
        return q;
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
    // Eight 16-bit values to a word of codes.  The quotient by the correctly rounded reciprocal
    // and one correction (Markstein, "Computation of elementary functions on the IBM RISC System
    // / 6000": it is the correctly rounded one), which leaves out what a division does for
    // numbers at the ends of the range; those go by the division.
    __device__ __forceinline__ uint32_t codes(const uint4 &w) const
    {
        constexpr float kMagic = 12582912.f;                                // 1.5 2^23: integers in its low bits
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        uint32_t d = 0;
        if (large || s < 1e-30f) {                                          // (zeros, and NaN among the values, too)
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                const uint32_t v = i < 2 ? u[0] : i < 4 ? u[1] : i < 6 ? u[2] : u[3];
                d |= code(i & 1 ? hi16<BF16>(v) : lo16<BF16>(v)) << (4 * i);
            }
            return d;
        }
        const float inv = __frcp_rn(s);
        const int base = static_cast<int>(z) - 0x4b400000;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = i & 1 ? hi16<BF16>(u[i / 2]) : lo16<BF16>(u[i / 2]);
            float q = __fmul_rn(x, inv);
            q = fmaf(fmaf(-q, s, x), inv, q);
            d += static_cast<uint32_t>(min(max(__float_as_int(__fadd_rn(q, kMagic)) + base, 0), 15)) << (4 * i);
        }
        return d;
    }
};

// PART: only some of a head's threads rotate (0 < rot < D); the others' values are copied.  A kernel of
// its own: with the choice in one, whole heads took 5 us more (8192 tokens of 80 heads).
template <int D, bool BF16, bool PART>
__global__ void __launch_bounds__(kThreads, 7)
kv4_append_kernel(const __grid_constant__ Kv4AppendParams p)
{
    constexpr int kItems = D / 16;                       // threads per head
    constexpr int kCols = kThreads / kItems;             // heads side by side
    constexpr int kGroups = D / kKv4Group;
    if (threadIdx.x == 0)
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const qmm_paged_kv &kv = p.kv;
    const int t = blockIdx.x;
    const int lane = threadIdx.x & 31;
    const int item = threadIdx.x % kItems, col = threadIdx.x / kItems;
    const int hq = p.q_heads, hk = kv.kv_heads;
    const int rot_items = p.rot / 16;
    const bool turn = item < rot_items;
    // the thread's two chunks of a head (8 values each)
    int c0 = 2 * item, c1 = 2 * item + 1;
    if (turn && !p.interleaved) {
        c0 = item;
        c1 = item + rot_items;
    }
    // Queries come first, kBatch heads at a time, then keys and values, in one row of 2 hk heads.
    // The first of both are under way before the rest is known.
    const uint16_t *qsrc = p.q + t * p.q_stride + col * D;
    uint4 qa[kBatch], qb[kBatch], ka = {}, kb = {};
    auto fetch_q = [&](int h) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (h + u * kCols < hq) {
                qa[u] = __ldcs(reinterpret_cast<const uint4 *>(qsrc + u * (kCols * D) + 8 * c0));
                qb[u] = __ldcs(reinterpret_cast<const uint4 *>(qsrc + u * (kCols * D) + 8 * c1));
            }
        qsrc += kBatch * kCols * D;
    };
    auto fetch_kv = [&](int h) {
        if (h < 2 * hk) {
            const uint16_t *src = h < hk ? p.k + t * p.k_stride + h * D : p.v + t * p.v_stride + (h - hk) * D;
            ka = __ldcs(reinterpret_cast<const uint4 *>(src + 8 * c0));
            kb = __ldcs(reinterpret_cast<const uint4 *>(src + 8 * c1));
        }
    };
    fetch_q(col);
    fetch_kv(col);
    uint64_t wa[4], wb[4];                               // the norm's weights
    auto weights = [&](const uint16_t *w) {
        if (w) {
            unpack8<BF16>(*reinterpret_cast<const uint4 *>(w + 8 * c0), wa);
            unpack8<BF16>(*reinterpret_cast<const uint4 *>(w + 8 * c1), wb);
        }
    };
    weights(p.q_norm);

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
    uint64_t cs[4], sn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        cs[i] = sn[i] = 0;
    if (turn) {
        const ulonglong2 *row = reinterpret_cast<const ulonglong2 *>(p.cos_sin + static_cast<long long>(pos) * p.rot + 8 * item);
        const ulonglong2 *rows = reinterpret_cast<const ulonglong2 *>(p.cos_sin + static_cast<long long>(pos) * p.rot +
                                                                      p.rot / 2 + 8 * item);
        const ulonglong2 u0 = row[0], u1 = row[1], w0 = rows[0], w1 = rows[1];
        cs[0] = u0.x; cs[1] = u0.y; cs[2] = u1.x; cs[3] = u1.y;
        sn[0] = w0.x; sn[1] = w0.y; sn[2] = w1.x; sn[3] = w1.y;
    }
    int page, slot;
    const bool place = find_slot(kv, p.by_page, seq, pos, p.status, page, slot);

    // (sums of rounded products: written as sums they came out fused, so they are products with
    // ones that the compiler does not know)
    const uint64_t plus = pair(p.one, p.one), minus = pair(-p.one, -p.one);
    // Norm and rotation of a head's chunks, rounded to the type.  The whole warp comes here together;
    // what its columns without a head hold does not matter.
    auto turned = [&](uint4 &a, uint4 &b, bool norm) {
        if (PART && !turn && !norm)
            return;                                      // the same bits
        uint64_t x[4], y[4];
        unpack8<BF16>(a, x);
        unpack8<BF16>(b, y);
        if (norm) {
            auto squares = [&] {
                uint64_t s2 = mul2(x[0], x[0]);
#pragma unroll
                for (int i = 1; i < 4; ++i)
                    s2 = fma2(x[i], x[i], s2);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s2 = fma2(y[i], y[i], s2);
                const float2 f = unpair(s2);
                float ss = f.x + f.y;
#pragma unroll
                for (int d = 1; d < kItems; d <<= 1)
                    ss += __shfl_xor_sync(0xffffffffu, ss, d);
                return ss;
            };
            float mean = fmaf(squares(), 1.f / D, p.eps);
            // bf16 heads whose squares leave fp32's range: times a power of two first
            if (BF16 && __any_sync(0xffffffffu, !(mean < 0x1p120f) || mean < 0x1p-80f)) {
                const float c = mean < 0x1p-80f ? 0x1p100f : mean < 0x1p120f ? 1.f : 0x1p-70f;
                const uint64_t c2 = pair(c, c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = mul2(x[i], c2);
                    y[i] = mul2(y[i], c2);
                }
                mean = fmaf(squares(), 1.f / D, p.eps * c * c);
            }
            const float r = rsqrtf(mean);
            const uint64_t r2 = pair(r, r);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = mul2(mul2(x[i], r2), wa[i]);
                y[i] = mul2(mul2(y[i], r2), wb[i]);
            }
        }
        if (p.rot > 0 && p.interleaved) {
            if (turn) {
                // pairs side by side
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint64_t &z = i < 4 ? x[i & 3] : y[i & 3];
                    const float2 cc = unpair(cs[i / 2]), ss = unpair(sn[i / 2]), f = unpair(z);
                    const float c = i & 1 ? cc.y : cc.x, s = i & 1 ? ss.y : ss.x;
                    z = pair(__fsub_rn(__fmul_rn(f.x, c), __fmul_rn(f.y, s)), __fadd_rn(__fmul_rn(f.y, c), __fmul_rn(f.x, s)));
                }
            }
        } else if (PART ? turn : p.rot > 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t x0 = x[i], y0 = y[i];
                x[i] = fma2(mul2(y0, sn[i]), minus, mul2(x0, cs[i]));
                y[i] = fma2(mul2(x0, sn[i]), plus, mul2(y0, cs[i]));
            }
        }
        a = pack8<BF16>(x);
        b = pack8<BF16>(y);
    };

    const int first = (threadIdx.x & ~31) / kItems;      // the warp's first column
    uint16_t *dst = p.q_out + (static_cast<long long>(t) * hq + col) * D;
    const bool work = p.rot > 0 || p.q_norm;
    for (int h0 = first; h0 < hq;) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (h0 + u * kCols >= hq)
                break;
            if (work)
                turned(qa[u], qb[u], p.q_norm != nullptr);
            if (h0 + u * kCols + (col - first) < hq) {
                *reinterpret_cast<uint4 *>(dst + u * (kCols * D) + 8 * c0) = qa[u];
                *reinterpret_cast<uint4 *>(dst + u * (kCols * D) + 8 * c1) = qb[u];
            }
        }
        dst += kBatch * kCols * D;
        h0 += kBatch * kCols;
        fetch_q(h0 + (col - first));
    }
    if (!place)
        return;
    const long long at = page * kv.page_stride + slot * kv.slot_stride;
    const long long sat = scale_offset(p.sc, page, slot);
    if (p.k_norm != p.q_norm)
        weights(p.k_norm);
    for (int h0 = first; h0 < 2 * hk; h0 += kCols) {
        const int h = h0 + (col - first);
        const bool is_k = h < hk;
        if (h0 < hk && (p.rot > 0 || p.k_norm)) {        // (a warp may hold keys and values side by side)
            uint4 a = ka, b = kb;
            turned(a, b, p.k_norm != nullptr);
            if (is_k) {
                ka = a;
                kb = b;
            }
        }
        // extremes of the groups, group g in half g of a word
        uint32_t lo0, hi0, lo1, hi1;
        extremes<BF16>(ka, lo0, hi0);
        extremes<BF16>(kb, lo1, hi1);
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
        // a thread works out one group's scale, its pair's first thread the first's
        const bool second = kGroups == 2 && item & 1;
        const Quant<BF16> mine(second ? hi16<BF16>(lo) : lo16<BF16>(lo), second ? hi16<BF16>(hi) : lo16<BF16>(hi));
        Quant<BF16> g0 = mine, g1 = mine;
        if constexpr (kGroups == 2) {
            const Quant<BF16> other = mine.swapped();
            g0 = second ? other : mine;
            g1 = second ? mine : other;
        }
        if (h < 2 * hk) {
            const uint32_t w0 = (kGroups == 2 && c0 >> 3 ? g1 : g0).codes(ka);
            const uint32_t w1 = (kGroups == 2 && c1 >> 3 ? g1 : g0).codes(kb);
            const int head = is_k ? h : h - hk;
            uint8_t *to = static_cast<uint8_t *>(is_k ? kv.k : kv.v) + at + head * kv.head_stride;
            *reinterpret_cast<uint32_t *>(to + 4 * c0) = w0;
            *reinterpret_cast<uint32_t *>(to + 4 * c1) = w1;
            if (item == 0) {
                uint16_t *sd = p.sc.base + sat + head * p.sc.head + (is_k ? 0 : kGroups);
                if constexpr (kGroups == 2)
                    *reinterpret_cast<uint32_t *>(sd) = g0.pattern | g1.pattern << 16;
                else
                    *sd = static_cast<uint16_t>(g0.pattern);
            }
        }
        fetch_kv(h + kCols);
    }
}

template <int D, bool BF16, bool PART>
cudaError_t launch_part(const Kv4AppendParams &p, cudaStream_t stream)
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
    return cudaLaunchKernelEx(&cfg, kv4_append_kernel<D, BF16, PART>, p);
}

template <int D, bool BF16>
cudaError_t launch_append(const Kv4AppendParams &p, cudaStream_t stream)
{
    return p.rot > 0 && p.rot < D ? launch_part<D, BF16, true>(p, stream) : launch_part<D, BF16, false>(p, stream);
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
