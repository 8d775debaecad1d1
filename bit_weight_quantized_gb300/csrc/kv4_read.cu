// kv4_read.cu -- reading the 4-bit paged cache back: (c - z) s for the last tokens of every
// sequence, or for all keys that a call's tokens see, exact in 16 bits.
//
// Bound by memory: 4.25 bits a value come in, 16 go out.  A thread turns sixteen codes into a
// 32-byte store (or two of 16, where the output is aligned to less), so that a warp's loads and
// stores are whole lines; a block finds the places of its tokens first, and has kFlight loads a
// thread under way.  131072 keys of 8 heads of 128: 103.6 us, 6.6 TB/s (eight codes and 16 bytes
// a thread 128; one load under way 116, four 111; sixteen tokens a block 106).
#include <algorithm>

#include "kv4.cuh"

namespace qmm {

namespace {

constexpr int kThreads = 256;
constexpr int kMostRows = 8;                             // tokens per block
constexpr int kFlight = 2;                               // loads in flight per thread

struct Place {
    long long codes, scales;                             // offsets of (page, slot), -1: nothing to read
};

// All heads' keys and values of `rows` places to rows of D, by the whole block.
template <int D, bool BF16, typename F>
__device__ __forceinline__ void convert(const Kv4ReadParams &p, const Place *places, int rows, F row_of)
{
    constexpr int kPieces = D / 16;                      // of a head
    constexpr int kGroups = D / kKv4Group;
    const qmm_paged_kv &kv = p.kv;
    // pieces of a token, 16 codes: [key, value][head][piece]
    const int all = rows * 2 * kv.kv_heads * kPieces;
    const int piece = threadIdx.x % kPieces;
    for (int e0 = threadIdx.x; e0 < all; e0 += kFlight * kThreads) {
        uint2 w[kFlight];
        uint32_t pattern[kFlight];
        uint16_t *dst[kFlight];
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int e = e0 + u * kThreads;
            dst[u] = nullptr;
            w[u] = make_uint2(0u, 0u);
            pattern[u] = 0;
            if (e < all) {
                const int row = p.by_heads(e / kPieces), i = row >> 1, head = e / kPieces - row * kv.kv_heads;
                const bool is_v = row & 1;
                const Place at = places[i];
                if (at.codes >= 0) {
                    const uint8_t *src = static_cast<const uint8_t *>(is_v ? kv.v : kv.k) + at.codes + head * kv.head_stride;
                    w[u] = __ldcs(reinterpret_cast<const uint2 *>(src) + piece);
                    pattern[u] = p.sc.base[at.scales + head * p.sc.head + (is_v ? kGroups : 0) + piece / 4];
                    dst[u] = row_of(i, head, is_v) + 16 * piece;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kFlight; ++u)
            if (dst[u]) {
                const GroupScale<BF16> sc(pattern[u]);
                const uint4 a = sc.values(w[u].x), b = sc.values(w[u].y);
                if (p.wide) {
                    asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst[u]), "r"(a.x),
                                 "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                                 : "memory");
                } else {
                    reinterpret_cast<uint4 *>(dst[u])[0] = a;
                    reinterpret_cast<uint4 *>(dst[u])[1] = b;
                }
            }
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads)
kv4_read_kernel(const __grid_constant__ Kv4ReadParams p)
{
    __shared__ Place places[kMostRows];
    if (threadIdx.x == 0)
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const qmm_paged_kv &kv = p.kv;
    const int t0 = blockIdx.x * p.rows, rows = min(p.rows, kv.tokens - t0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = warp; i < rows; i += kThreads / 32) {
        int seq = 0, end = 0, keys = 0;
        find_sequence(kv, t0 + i, lane, seq, end, keys);
        if (lane == 0) {
            Place at = {-1, -1};
            const int pos = seq < kv.batch ? max(keys, 0) - (end - (t0 + i)) : -1;
            if (pos >= table_keys(kv)) {
                record_error(p.status, QMM_ERR_INDEX);
            } else if (pos >= 0) {                       // (negative: padding)
                int page, slot;
                if (find_slot(kv, p.by_page, seq, pos, p.status, page, slot)) {
                    at.codes = page * kv.page_stride + slot * kv.slot_stride;
                    at.scales = scale_offset(p.sc, page, slot);
                }
            }
            places[i] = at;
        }
    }
    __syncthreads();
    convert<D, BF16>(p, places, rows, [&](int i, int head, bool is_v) {
        return (is_v ? p.v : p.k) + (static_cast<long long>(t0 + i) * kv.kv_heads + head) * D;
    });
}

// The keys of a sequence that the call's new tokens see, in 16 bits: blocks (x, y) take p.rows
// keys of sequence y at a time.  Keys lie [sequence][head][p.cap keys][D], a page per sequence to
// attn_chunk.cuh, whose block table is written here, too.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads)
kv4_unpack_kernel(const __grid_constant__ Kv4ReadParams p)
{
    __shared__ Place places[kMostRows];
    if (threadIdx.x == 0)
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const qmm_paged_kv &kv = p.kv;
    const int b = blockIdx.y;
    if (blockIdx.x == 0 && threadIdx.x == 0)
        p.table[b] = b;
    const int count = kv.kv_len[b], tokens = seq_tokens(kv, b).y;
    if (tokens == 0)
        return;
    // (zeros for keys past the table: the length that is wrong is recorded, and what follows
    // reads nothing but what was written here)
    const int known = seq_keys(kv, count, p.status), keys = min(count, p.cap);
    const int lo = p.window > 0 ? window_start(keys - tokens, p.window) : 0;
    for (long long from = lo + static_cast<long long>(blockIdx.x) * p.rows; from < keys; from += static_cast<long long>(gridDim.x) * p.rows) {
        const int key0 = static_cast<int>(from), rows = min(p.rows, keys - key0);
        __syncthreads();                                 // the last keys' places have been read
        if (static_cast<int>(threadIdx.x) < rows) {
            Place at = {-1, -1};
            int page, slot;
            const int key = key0 + threadIdx.x;
            if (key < known && find_slot(kv, p.by_page, b, key, p.status, page, slot)) {
                at.codes = page * kv.page_stride + slot * kv.slot_stride;
                at.scales = scale_offset(p.sc, page, slot);
            }
            places[threadIdx.x] = at;
        }
        __syncthreads();
        convert<D, BF16>(p, places, rows, [&](int i, int head, bool is_v) {
            return (is_v ? p.v : p.k) + ((static_cast<long long>(b) * kv.kv_heads + head) * p.cap + key0 + i) * D;
        });
    }
}

template <int D, bool BF16>
cudaError_t launch_read(const Kv4ReadParams &p, int num_sms, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    // (p.cap may be far above the keys there are: no more blocks than some waves of them)
    cfg.gridDim = p.table ? dim3(std::min((p.cap + p.rows - 1) / p.rows, std::max(1, 32 * num_sms / p.kv.batch)), p.kv.batch)
                          : dim3((p.kv.tokens + p.rows - 1) / p.rows);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return p.table ? cudaLaunchKernelEx(&cfg, kv4_unpack_kernel<D, BF16>, p) : cudaLaunchKernelEx(&cfg, kv4_read_kernel<D, BF16>, p);
}

}  // namespace

cudaError_t launch_kv4_read(Kv4ReadParams &p, int num_sms, cudaStream_t stream)
{
    p.rows = p.table ? kMostRows : std::max(1, std::min(kMostRows, p.kv.tokens / (4 * num_sms)));
    // the words of a block's tokens are counted in 32 bits
    while (p.rows > 1 && static_cast<long long>(p.rows) * p.kv.kv_heads > (1 << 24))
        p.rows /= 2;
    p.wide = (reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v)) % 32 == 0;
    const bool bf16 = p.kv.dtype == QMM_BF16;
    if (p.kv.head_dim == 128)
        return bf16 ? launch_read<128, true>(p, num_sms, stream) : launch_read<128, false>(p, num_sms, stream);
    return bf16 ? launch_read<64, true>(p, num_sms, stream) : launch_read<64, false>(p, num_sms, stream);
}

}  // namespace qmm
