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
constexpr int kFlight = 2, kAhead = 4;                   // loads in flight per thread

struct Place {
    long long codes, scales;                             // offsets of (page, slot), -1: nothing to read
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads)
kv4_read_kernel(const __grid_constant__ Kv4ReadParams p)
{
    constexpr int kPieces = D / 16;                      // of a head
    constexpr int kGroups = D / kKv4Group;
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
                    dst[u] = (is_v ? p.v : p.k) + (static_cast<long long>(t0 + i) * kv.kv_heads + head) * D + 16 * piece;
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

// The keys of a sequence that the call's new tokens see, in 16 bits: blocks (x, y) take kMostRows
// keys of sequence y at a time.  Keys lie [sequence][head][p.cap keys][D], a page per sequence to
// attn_chunk.cuh, whose block table is written here, too.  A thread keeps a key and a piece of 16
// values and goes through the heads.  Bound by latency (lengths and page, codes, stores: 16.6 us
// for 16384 keys of 8 heads alone, where memory would take 3 and L2 10); with the lengths, then
// the page, then two loads at a time 17.4.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads)
kv4_unpack_kernel(const __grid_constant__ Kv4ReadParams p)
{
    constexpr int kPieces = D / 16, kGroups = D / kKv4Group;
    constexpr int kSide = kThreads / (kPieces * kMostRows);          // heads side by side
    if (threadIdx.x == 0)
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const qmm_paged_kv &kv = p.kv;
    const int b = blockIdx.y, heads = kv.kv_heads;
    if (blockIdx.x == 0 && threadIdx.x == 0)
        p.table[b] = b;
    // (pages are looked up beside the lengths, and ahead)
    const int piece = threadIdx.x % kPieces, side = threadIdx.x / (kPieces * kMostRows), most = table_keys(kv);
    const long long step = static_cast<long long>(gridDim.x) * kMostRows;
    const int32_t *row = kv.block_table + static_cast<long long>(b) * kv.blocks;
    auto page_of = [&](long long key) { return key < most ? row[p.by_page(static_cast<int>(key))] : -1; };
    long long key = static_cast<long long>(blockIdx.x) * kMostRows + threadIdx.x / kPieces % kMostRows;
    const int count = kv.kv_len[b], tokens = seq_tokens(kv, b).y;
    if (p.window > 0)
        key += window_start(min(max(count, 0), p.cap) - tokens, p.window);
    int page = page_of(key), next;
    if (tokens == 0)
        return;
    // (zeros for keys past the table and of pages that are not there: what is wrong is recorded,
    // and what follows reads nothing but what was written here)
    const int known = seq_keys(kv, count, p.status), keys = min(count, p.cap);
    for (; key < keys; key += step, page = next) {
        next = page_of(key + step);
        bool in = key < known;
        if (in && (page < 0 || page >= kv.num_pages)) {
            record_error(p.status, QMM_ERR_INDEX);
            in = false;
        }
        const int slot = static_cast<int>(key) - p.by_page(static_cast<int>(key)) * kv.page_size;
        const long long at = in ? page * kv.page_stride + slot * kv.slot_stride + 8 * piece : 0;
        const uint16_t *pattern_at = p.sc.base + (in ? scale_offset(p.sc, page, slot) + piece / 4 : 0);
        const long long head = static_cast<long long>(p.cap) * D, to = b * heads * head + key * D + 16 * piece;
        // keys' heads and then values', kAhead loads under way
        for (int e0 = side; e0 < 2 * heads; e0 += kAhead * kSide) {
            uint2 w[kAhead];
            uint32_t pattern[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int e = e0 + u * kSide, h = e < heads ? e : e - heads;
                w[u] = make_uint2(0u, 0u);
                pattern[u] = 0;
                if (in && e < 2 * heads) {
                    const uint8_t *src = static_cast<const uint8_t *>(e < heads ? kv.k : kv.v) + at + h * kv.head_stride;
                    w[u] = __ldcs(reinterpret_cast<const uint2 *>(src));
                    pattern[u] = pattern_at[(e < heads ? 0 : kGroups) + h * p.sc.head];
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int e = e0 + u * kSide;
                if (e >= 2 * heads)
                    break;
                const GroupScale<BF16> sc(pattern[u]);
                const uint4 x = sc.values(w[u].x), y = sc.values(w[u].y);
                uint16_t *dst = e < heads ? p.k + to + e * head : p.v + to + (e - heads) * head;
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(x.x), "r"(x.y),
                             "r"(x.z), "r"(x.w), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w)
                             : "memory");
            }
        }
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
