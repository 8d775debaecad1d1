// kv4_read.cu -- reading the 4-bit paged cache back: (c - z) s for the last tokens of every
// sequence, exact in 16 bits.
//
// Bound by memory: 4.25 bits a value come in, 16 go out.  A thread turns eight codes (a
// word) into a 16-byte store, so that a warp's loads and stores are whole lines; a block
// finds the places of its tokens first, and takes four words a thread at a time.
#include <algorithm>

#include "kv4.cuh"

namespace qmm {

namespace {

constexpr int kThreads = 256;
constexpr int kMostRows = 16;                            // tokens per block
constexpr int kFlight = 4;                               // words in flight per thread

struct Place {
    long long codes, scales;                             // offsets of (page, slot), -1: nothing to read
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads)
kv4_read_kernel(const __grid_constant__ Kv4ReadParams p)
{
    constexpr int kWords = D / 8;                        // words of codes per head
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
    // words of a token: [key, value][head][word]
    const int per = 2 * kv.kv_heads * kWords, all = rows * per;
    const int word = threadIdx.x % kWords;
    for (int e0 = threadIdx.x; e0 < all; e0 += kFlight * kThreads) {
        uint32_t w[kFlight], pattern[kFlight];
        uint16_t *dst[kFlight];
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int e = e0 + u * kThreads;
            dst[u] = nullptr;
            w[u] = pattern[u] = 0;
            if (e < all) {
                // (token, key or value, head): e / kWords in the heads' base
                const int row = p.by_heads(e / kWords), i = row >> 1, head = e / kWords - row * kv.kv_heads;
                const bool is_v = row & 1;
                const Place at = places[i];
                if (at.codes >= 0) {
                    const uint8_t *src = static_cast<const uint8_t *>(is_v ? kv.v : kv.k) + at.codes + head * kv.head_stride;
                    w[u] = __ldcs(reinterpret_cast<const uint32_t *>(src) + word);
                    pattern[u] = p.sc.base[at.scales + head * p.sc.head + (is_v ? kGroups : 0) + (word >> 3)];
                    dst[u] = (is_v ? p.v : p.k) + (static_cast<long long>(t0 + i) * kv.kv_heads + head) * D + 8 * word;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kFlight; ++u)
            if (dst[u])
                __stcs(reinterpret_cast<uint4 *>(dst[u]), GroupScale<BF16>(pattern[u]).values(w[u]));
    }
}

template <int D, bool BF16>
cudaError_t launch_read(const Kv4ReadParams &p, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((p.kv.tokens + p.rows - 1) / p.rows);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4_read_kernel<D, BF16>, p);
}

}  // namespace

cudaError_t launch_kv4_read(Kv4ReadParams &p, int num_sms, cudaStream_t stream)
{
    p.rows = std::max(1, std::min(kMostRows, p.kv.tokens / (4 * num_sms)));
    // the words of a block's tokens are counted in 32 bits
    while (p.rows > 1 && static_cast<long long>(p.rows) * p.kv.kv_heads > (1 << 24))
        p.rows /= 2;
    const bool bf16 = p.kv.dtype == QMM_BF16;
    if (p.kv.head_dim == 128)
        return bf16 ? launch_read<128, true>(p, stream) : launch_read<128, false>(p, stream);
    return bf16 ? launch_read<64, true>(p, stream) : launch_read<64, false>(p, stream);
}

}  // namespace qmm
