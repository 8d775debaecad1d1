// api.cu -- the C ABI of libqmm (include/qmm.h): argument checks, device
// facts, TMA descriptors and dispatch to the kernels.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "decode.h"
#include "gemv.h"
#include "w4a8.h"
#include "gemm.h"
#include "kv4.h"
#include "paged.h"

namespace qmm {

// The library's device status word (one per device that loads the library).
__device__ int g_status_word = 0;

// One warp waits on an mbarrier that nothing arrives at; the bounded wait gives
// up, records QMM_ERR_TIMEOUT and the kernel returns.
__global__ void watchdog_selftest_kernel(int *status)
{
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_barrier_init();
    }
    __syncwarp();
    mbar_wait(&bar, 0, status);
}

namespace {

constexpr int kMaxDevices = 64;

struct DeviceFacts {
    bool ready = false;
    qmm_status usable = QMM_ERR_DEVICE;
    int num_sms = 0;
    int smem_optin = 0;
    int smem_pair = 0;   // per-CTA shared memory with which two CTAs share an SM
    int *status = nullptr;
};

DeviceFacts g_facts[kMaxDevices];
std::mutex g_mutex;
std::atomic<int> g_gemv_kernel{QMM_GEMV_AUTO};

// Facts about the current device, computed once per device.
const DeviceFacts *device_facts()
{
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return nullptr;
    }
    std::lock_guard<std::mutex> lock(g_mutex);
    DeviceFacts &f = g_facts[dev];
    if (!f.ready) {
        int major = 0, minor = 0;
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
        cudaDeviceGetAttribute(&f.num_sms, cudaDevAttrMultiProcessorCount, dev);
        cudaDeviceGetAttribute(&f.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
        int smem_sm = 0, reserved = 0;
        cudaDeviceGetAttribute(&smem_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
        cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev);
        f.smem_pair = (smem_sm / 2 - reserved) / 128 * 128;
        void *addr = nullptr;
        cudaError_t e = cudaGetSymbolAddress(&addr, g_status_word);
        if (e != cudaSuccess || major != 10 || minor != 3 || f.num_sms <= 0) {
            cudaGetLastError();
            f.usable = QMM_ERR_DEVICE;
        } else {
            f.status = static_cast<int *>(addr);
            f.usable = QMM_OK;
        }
        f.ready = true;
    }
    return &f;
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        else
            cudaGetLastError();
    });
    return fn;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

qmm_status from_cuda(cudaError_t e) { return e == cudaSuccess ? QMM_OK : QMM_ERR_CUDA; }

}  // namespace

// 2-D tensor map over a byte matrix [rows][row_bytes] with a box of
// box_cols bytes x box_rows rows.  Returns false if the driver refuses it.
bool encode_byte_tmap(CUtensorMap *map, const void *base, long long row_bytes, long long rows,
                      int box_cols, int box_rows, bool swizzle128)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc)
        return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims,
                     strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// 2-D tensor map over a 16-bit matrix [rows][cols] (elements) with the
// 128-byte swizzle, box box_cols x box_rows elements.
bool encode_u16_tmap(CUtensorMap *map, const void *base, long long cols, long long rows,
                     int box_cols, int box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc)
        return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols * 2)};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void *>(base), dims,
                     strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

bool encode_u64_tmap(CUtensorMap *map, const void *base, long long cols, long long rows,
                     int box_cols, int box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc)
        return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols * 8)};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT64, 2, const_cast<void *>(base), dims,
                     strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

void attn_set_tma(AttnParams &p)
{
    p.box = 0;
    // one index for page and head: the page stride in head strides
    long long step = 1, stride = p.kv.page_stride;
    if (p.kv.kv_heads > 1) {
        stride = p.kv.head_stride;
        if (stride <= 0 || p.kv.page_stride % stride)
            return;
        step = p.kv.page_stride / stride;
    }
    // a box lies in one page and in one 128-key tile, and is whole 8-row groups of
    // the swizzle: the largest power of two in both, at least 8
    int box = 128;
    while (p.kv.page_size % box)
        box /= 2;
    const long long rows = (p.kv.num_pages - 1LL) * step + p.kv.kv_heads;
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (box < 8 || !enc || p.kv.num_pages < 1 || step < 1 || rows > 0x7fffffffLL)
        return;
    const cuuint64_t dims[5] = {64, 8, static_cast<cuuint64_t>(p.kv.head_dim / 64),
                                static_cast<cuuint64_t>(p.kv.page_size / 8), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[4] = {static_cast<cuuint64_t>(p.kv.slot_stride) * 2, 128,
                                   static_cast<cuuint64_t>(p.kv.slot_stride) * 16, static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t boxes[5] = {64, 8, static_cast<cuuint32_t>(p.kv.head_dim / 64), static_cast<cuuint32_t>(box / 8), 1};
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    CUtensorMap *maps[2] = {&p.tmk, &p.tmv};
    void *const base[2] = {p.kv.k, p.kv.v};
    for (int i = 0; i < 2; ++i)
        if (enc(maps[i], CU_TENSOR_MAP_DATA_TYPE_UINT16, 5, base[i], dims, strides, boxes, one,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return;
    p.box = box;
    p.page_step = static_cast<int>(step);
}

bool attn_set_q_tma(AttnParams &p)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    // (a single token's stride is not looked at)
    const long long stride = p.kv.tokens > 1 ? p.q_stride : static_cast<long long>(p.q_heads) * p.kv.head_dim;
    if (!enc || p.group > 128 || stride <= 0)
        return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.kv.head_dim), static_cast<cuuint64_t>(p.q_heads),
                                static_cast<cuuint64_t>(p.kv.tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(p.kv.head_dim) * 2, static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(128 / p.group)};
    const cuuint32_t one[3] = {1, 1, 1};
    return enc(&p.tmq, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<uint16_t *>(p.q), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

void skinny_set_tma(GemvParams &p)
{
    p.tma = 0;
    if (p.use_bulk && p.pitch % 16 == 0 && p.pitch > 0 && p.pitch <= 2048 && p.row_bytes % 16 == 0 &&
        p.seg_bytes % 16 == 0 && p.rb >= 1 && p.rb <= 256 &&
        static_cast<long long>(p.stage_bytes) >= static_cast<long long>(p.rb) * p.pitch &&
        encode_u64_tmap(&p.tmw, p.packed, p.row_bytes / 8, p.N, p.pitch / 8, p.rb))
        p.tma = 1;
}

// Shared checks of qmm_gemv / qmm_gemm (everything that needs no device).
static qmm_status check_qmm_args(const void *x, const uint8_t *packed, int bits, int group,
                                 const void *scales, int zero_const, const uint8_t *zeros,
                                 void *y, int M, int N, int K)
{
    if (M < 0 || N < 0 || K < 0)
        return QMM_ERR_SHAPE;
    if (bits < 1 || bits > 8)
        return QMM_ERR_BITS;
    if (group != 32 && group != 64 && group != 128)
        return QMM_ERR_SHAPE;
    if (K % group)
        return QMM_ERR_SHAPE;
    if (!zeros && (zero_const < 0 || zero_const > 255))
        return QMM_ERR_SHAPE;
    if (M == 0 || N == 0)
        return QMM_OK;
    if (!y)
        return QMM_ERR_NULL;
    if (K == 0)
        return QMM_OK;
    if (!x || !packed || !scales)
        return QMM_ERR_NULL;
    if (!aligned(x, 16) || !aligned(packed, 4) || !aligned(scales, 2) || !aligned(y, 2))
        return QMM_ERR_ALIGN;
    return QMM_OK;
}

// Shared checks of the paged cache calls (everything that needs no device).  A
// batch without tokens or sequences passes with the sizes alone.
static qmm_status check_paged(const qmm_paged_kv *kv)
{
    if (!kv)
        return QMM_ERR_NULL;
    if (kv->batch < 0 || kv->tokens < 0 || kv->num_pages < 0 || kv->page_size < 1 || kv->blocks < 0 ||
        kv->kv_heads < 1 || kv->head_dim < 1)
        return QMM_ERR_SHAPE;
    if (kv->dtype != QMM_F16 && kv->dtype != QMM_BF16)
        return QMM_ERR_UNSUPPORTED;
    if (kv->head_dim != 64 && kv->head_dim != 128)
        return QMM_ERR_UNSUPPORTED;
    // a stride counts only where there is more than one of what it separates
    if ((kv->num_pages > 1 && kv->page_stride < 0) || (kv->page_size > 1 && kv->slot_stride < 0) ||
        (kv->kv_heads > 1 && kv->head_stride < 0))
        return QMM_ERR_SHAPE;
    if ((kv->num_pages > 1 && kv->page_stride % 8) || (kv->page_size > 1 && kv->slot_stride % 8) ||
        (kv->kv_heads > 1 && kv->head_stride % 8))
        return QMM_ERR_ALIGN;
    if (kv->batch == 0 || kv->tokens == 0)
        return QMM_OK;
    if (!kv->cu_q || !kv->kv_len || (kv->blocks > 0 && !kv->block_table) ||
        (kv->blocks > 0 && kv->num_pages > 0 && (!kv->k || !kv->v)))
        return QMM_ERR_NULL;
    if (!aligned(kv->k, 16) || !aligned(kv->v, 16) || !aligned(kv->block_table, 4) || !aligned(kv->cu_q, 4) ||
        !aligned(kv->kv_len, 4))
        return QMM_ERR_ALIGN;
    return QMM_OK;
}

// Shared checks of the 4-bit cache calls; fills what the kernels take.  A batch without tokens
// or sequences passes with the sizes alone.
static qmm_status check_kv4(const qmm_paged_kv4 *kv, qmm_paged_kv *codes, Kv4Scales *sc)
{
    if (!kv)
        return QMM_ERR_NULL;
    // (the members up to dtype are qmm_paged_kv's; strides of 16 bytes pass as multiples of 8)
    *codes = {kv->k, kv->v, kv->page_stride, kv->slot_stride, kv->head_stride, kv->block_table, kv->cu_q, kv->kv_len,
              kv->num_pages, kv->page_size, kv->blocks, kv->batch, kv->tokens, kv->kv_heads, kv->head_dim, kv->dtype};
    *sc = {static_cast<uint16_t *>(kv->scales), kv->scale_page_stride, kv->scale_slot_stride, kv->scale_head_stride};
    if (const qmm_status st = check_paged(codes); st != QMM_OK)
        return st;
    if (kv->kv_heads > 65536)
        return QMM_ERR_UNSUPPORTED;
    // (the kernels multiply page and slot numbers by 32-bit strides)
    const int64_t most = 0x7fffffff, slots = kv->page_size - 1, heads = kv->kv_heads - 1;
    if ((kv->num_pages > 1 && (kv->page_stride > most || sc->page > most)) ||
        (slots > 0 && (kv->slot_stride > most / slots || sc->slot > most / slots)) ||
        (heads > 0 && (kv->head_stride > most || sc->head > most)))
        return QMM_ERR_UNSUPPORTED;
    if ((kv->num_pages > 1 && sc->page < 0) || (kv->page_size > 1 && sc->slot < 0) || (kv->kv_heads > 1 && sc->head < 0))
        return QMM_ERR_SHAPE;
    const int step = kv->head_dim / 32;   // a key's scale patterns
    if ((kv->num_pages > 1 && (kv->page_stride % 16 || sc->page % step)) ||
        (kv->page_size > 1 && (kv->slot_stride % 16 || sc->slot % step)) ||
        (kv->kv_heads > 1 && (kv->head_stride % 16 || sc->head % step)))
        return QMM_ERR_ALIGN;
    if (kv->batch == 0 || kv->tokens == 0)
        return QMM_OK;
    if (kv->blocks > 0 && kv->num_pages > 0 && !kv->scales)
        return QMM_ERR_NULL;
    if (!aligned(kv->scales, 2 * step))
        return QMM_ERR_ALIGN;
    return QMM_OK;
}

}  // namespace qmm

using namespace qmm;

extern "C" {

int qmm_abi_version(void) { return QMM_ABI_VERSION; }

const char *qmm_status_string(qmm_status s)
{
    switch (s) {
    case QMM_OK: return "ok";
    case QMM_ERR_NULL: return "a required pointer is NULL";
    case QMM_ERR_BITS: return "bits outside the supported range";
    case QMM_ERR_SHAPE: return "invalid shape or group size";
    case QMM_ERR_ALIGN: return "pointer or pitch breaks an alignment rule";
    case QMM_ERR_UNSUPPORTED: return "valid request that is not implemented";
    case QMM_ERR_CUDA: return "CUDA runtime or launch failure";
    case QMM_ERR_TIMEOUT: return "device watchdog expired";
    case QMM_ERR_DEVICE: return "no usable sm_103a device";
    case QMM_ERR_INDEX: return "an index in device memory is out of range";
    }
    return "unknown status";
}

qmm_status qmm_pack(const uint8_t *codes, uint8_t *packed, int N, int K, int bits,
                    int32_t *bad_count, cudaStream_t stream)
{
    if (bits < 1 || bits > 8)
        return QMM_ERR_BITS;
    if (N < 0 || K < 0 || (static_cast<long long>(K) * bits) % 8)
        return QMM_ERR_SHAPE;
    if (N == 0 || K == 0)
        return QMM_OK;
    if (!codes || !packed)
        return QMM_ERR_NULL;
    if (bad_count && !aligned(bad_count, 4))
        return QMM_ERR_ALIGN;
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return QMM_ERR_DEVICE;
    return from_cuda(launch_pack(codes, packed, N, K, bits, bad_count, stream, f->num_sms));
}

qmm_status qmm_unpack(const uint8_t *packed, uint8_t *codes, int N, int K, int bits,
                      cudaStream_t stream)
{
    if (bits < 1 || bits > 8)
        return QMM_ERR_BITS;
    if (N < 0 || K < 0 || (static_cast<long long>(K) * bits) % 8)
        return QMM_ERR_SHAPE;
    if (N == 0 || K == 0)
        return QMM_OK;
    if (!codes || !packed)
        return QMM_ERR_NULL;
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return QMM_ERR_DEVICE;
    return from_cuda(launch_unpack(packed, codes, N, K, bits, stream, f->num_sms));
}

qmm_status qmm_gemv_float(const void *x, const uint8_t *packed, int ebits, int mbits, int group,
                          const void *scales, void *y, int M, int N, int K, cudaStream_t stream)
{
    if (ebits < 1 || mbits < 0 || 1 + ebits + mbits < 2 || 1 + ebits + mbits > 8)
        return QMM_ERR_BITS;
    if (M < 0 || N < 0 || K < 0 || M > 16)
        return QMM_ERR_SHAPE;
    if (group != 32 && group != 64 && group != 128)
        return QMM_ERR_SHAPE;
    if (K % group)
        return QMM_ERR_SHAPE;
    if (M == 0 || N == 0)
        return QMM_OK;
    if (!y)
        return QMM_ERR_NULL;
    if (K > 0 && (!x || !packed || !scales))
        return QMM_ERR_NULL;
    if (!aligned(x, 16) || !aligned(packed, 4) || !aligned(scales, 2) || !aligned(y, 2))
        return QMM_ERR_ALIGN;
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return QMM_ERR_DEVICE;
    if (K == 0)
        return from_cuda(cudaMemsetAsync(y, 0, static_cast<size_t>(M) * N * 2, stream));
    // codes with at most 4 exponent bits are exact fp16 numbers (times a power
    // of two; a 5-bit exponent field of 31 would read as inf): the decode
    // kernel runs them on the tensor cores
    const int bits = 1 + ebits + mbits;
    DecodePlan plan;
    if (ebits <= 4 && aligned(packed, 16) &&
        decode_plan(M, N, K, group, bits, false, false, f->num_sms, f->smem_pair, f->smem_optin, &plan)) {
        DecodeParams d;
        std::memset(&d, 0, sizeof(d));
        d.x = static_cast<const uint16_t *>(x);
        d.packed = packed;
        d.scales = static_cast<const uint16_t *>(scales);
        d.zeros = nullptr;
        d.y = y;
        d.status = f->status;
        d.row_bytes = static_cast<long long>(K) * bits / 8;
        d.M = M;
        d.N = N;
        d.K = K;
        d.group_log2 = group == 64 ? 6 : 7;
        d.zero_const = 0;
        d.ebits = ebits;
        d.mbits = mbits;
        d.fscale = static_cast<float>(1 << (15 - ((1 << (ebits - 1)) - 1)));
        d.pl = plan;
        decode_set_tma(d);
        return from_cuda(launch_decode_float(d, bits, stream));
    }
    return from_cuda(launch_gemv_fp(static_cast<const uint16_t *>(x), packed, ebits, mbits, group,
                                    static_cast<const uint16_t *>(scales), static_cast<uint16_t *>(y), M, N,
                                    K, stream));
}

qmm_status qmm_flip_sign(uint8_t *packed, int N, int K, int bits, cudaStream_t stream)
{
    if (bits < 1 || bits > 8)
        return QMM_ERR_BITS;
    if (N < 0 || K < 0 || (static_cast<long long>(K) * bits) % 8)
        return QMM_ERR_SHAPE;
    if (N == 0 || K == 0)
        return QMM_OK;
    if (!packed)
        return QMM_ERR_NULL;
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return QMM_ERR_DEVICE;
    return from_cuda(launch_flip_sign(packed, N, K, bits, stream, f->num_sms));
}

qmm_status qmm_gemv(const void *x, qmm_dtype x_dtype, const uint8_t *packed, int bits,
                    int group, const void *scales, const uint8_t *zeros, int zero_const,
                    void *y, qmm_dtype y_dtype, int M, int N, int K, cudaStream_t stream)
{
    qmm_status st = check_qmm_args(x, packed, bits, group, scales, zero_const, zeros, y, M, N, K);
    if (st != QMM_OK)
        return st;
    if (M > 16)
        return QMM_ERR_SHAPE;
    if ((x_dtype != QMM_F16 && x_dtype != QMM_BF16) || (y_dtype != QMM_F16 && y_dtype != QMM_BF16))
        return QMM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0)
        return QMM_OK;
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return QMM_ERR_DEVICE;
    if (K == 0)
        return from_cuda(cudaMemsetAsync(y, 0, static_cast<size_t>(M) * N * 2, stream));
    DecodePlan plan;
    if (g_gemv_kernel.load(std::memory_order_relaxed) == QMM_GEMV_AUTO && aligned(packed, 16) &&
        decode_plan(M, N, K, group, bits, zeros != nullptr, false, f->num_sms, f->smem_pair, f->smem_optin,
                    &plan)) {
        DecodeParams d;
        std::memset(&d, 0, sizeof(d));
        d.x = static_cast<const uint16_t *>(x);
        d.packed = packed;
        d.scales = static_cast<const uint16_t *>(scales);
        d.zeros = zeros;
        d.y = y;
        d.status = f->status;
        d.row_bytes = static_cast<long long>(K) * bits / 8;
        d.M = M;
        d.N = N;
        d.K = K;
        d.group_log2 = group == 64 ? 6 : 7;
        d.y_bf16 = y_dtype == QMM_BF16;
        d.x_bf16 = x_dtype == QMM_BF16;
        d.zero_const = zeros ? 0 : zero_const;
        d.vec_sz = aligned(scales, 16) && (!zeros || aligned(zeros, 8));
        d.pl = plan;
        decode_set_tma(d);
        return from_cuda(launch_decode(d, bits, false, stream));
    }

    if (x_dtype != QMM_F16)   // the skinny kernel stages fp16 activations only
        return QMM_ERR_UNSUPPORTED;
    GemvParams p;
    std::memset(&p, 0, sizeof(p));
    p.x = static_cast<const uint16_t *>(x);
    p.packed = packed;
    p.scales = static_cast<const uint16_t *>(scales);
    p.zeros = zeros;
    p.y = y;
    p.status = f->status;
    p.row_bytes = static_cast<long long>(K) * bits / 8;
    p.M = M;
    p.N = N;
    p.K = K;
    p.group = group;
    p.ng = K / group;
    p.zero_const = zeros ? 0 : zero_const;
    p.y_bf16 = y_dtype == QMM_BF16;
    int grid = 0, smem = 0;
    st = skinny_plan(p, bits, f->num_sms, f->smem_optin, f->smem_pair, &grid, &smem);
    if (st != QMM_OK)
        return st;
    p.use_bulk = aligned(packed, 16) && p.row_bytes % 16 == 0;
    skinny_set_tma(p);
    cudaError_t e;
    switch (bits) {
    case 1: e = gemv_launch_w1(p, grid, smem, stream); break;
    case 2: e = gemv_launch_w2(p, grid, smem, stream); break;
    case 3: e = gemv_launch_w3(p, grid, smem, stream); break;
    case 4: e = gemv_launch_w4(p, grid, smem, stream); break;
    case 5: e = gemv_launch_w5(p, grid, smem, stream); break;
    case 6: e = gemv_launch_w6(p, grid, smem, stream); break;
    case 7: e = gemv_launch_w7(p, grid, smem, stream); break;
    default: e = gemv_launch_w8(p, grid, smem, stream); break;
    }
    return from_cuda(e);
}

int qmm_gemv_route(int M, int N, int K, int bits, int group, int stored_zeros)
{
    if (M < 1 || M > 16 || N < 1 || K < 1 || bits < 1 || bits > 8 ||
        (group != 32 && group != 64 && group != 128) || K % group)
        return -static_cast<int>(QMM_ERR_SHAPE);
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return -static_cast<int>(QMM_ERR_DEVICE);
    if (g_gemv_kernel.load(std::memory_order_relaxed) != QMM_GEMV_AUTO)
        return QMM_GEMV_SKINNY;
    DecodePlan plan;
    return decode_plan(M, N, K, group, bits, stored_zeros != 0, false, f->num_sms, f->smem_pair, f->smem_optin,
                       &plan)
               ? QMM_GEMV_AUTO
               : QMM_GEMV_SKINNY;
}

size_t qmm_repack_bytes(int N, int K, int bits, int layout)
{
    if (N < 0 || K < 0 || bits < 1 || bits > 8)
        return 0;
    if (layout == QMM_LAYOUT_TILE16)
        return K % 64 ? 0 : static_cast<size_t>((N + 15) / 16) * 16 * K * bits / 8;
    if (layout == QMM_LAYOUT_INTERLEAVE4)
        return bits != 4 || K % 8 ? 0 : static_cast<size_t>(N) * K / 2;
    return 0;
}

qmm_status qmm_repack(const uint8_t *packed, uint8_t *out, int N, int K, int bits, int layout, cudaStream_t stream)
{
    if (bits < 1 || bits > 8)
        return QMM_ERR_BITS;
    if (N < 0 || K < 0 || (layout != QMM_LAYOUT_TILE16 && layout != QMM_LAYOUT_INTERLEAVE4))
        return QMM_ERR_SHAPE;
    if ((layout == QMM_LAYOUT_TILE16 && K % 64) || (layout == QMM_LAYOUT_INTERLEAVE4 && (bits != 4 || K % 8)))
        return QMM_ERR_SHAPE;
    if (N == 0 || K == 0)
        return QMM_OK;
    if (!packed || !out)
        return QMM_ERR_NULL;
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return QMM_ERR_DEVICE;
    return from_cuda(launch_repack(packed, out, N, K, bits, layout, stream, f->num_sms));
}

qmm_status qmm_gemv_tile16(const void *x, qmm_dtype x_dtype, const uint8_t *tiled, int bits, int group,
                           const void *scales, const uint8_t *zeros, int zero_const, void *y, qmm_dtype y_dtype,
                           int M, int N, int K, cudaStream_t stream)
{
    qmm_status st = check_qmm_args(x, tiled, bits, group, scales, zero_const, zeros, y, M, N, K);
    if (st != QMM_OK)
        return st;
    if (M > 16)
        return QMM_ERR_SHAPE;
    if ((x_dtype != QMM_F16 && x_dtype != QMM_BF16) || (y_dtype != QMM_F16 && y_dtype != QMM_BF16))
        return QMM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0)
        return QMM_OK;
    if (K > 0 && !aligned(tiled, 16))
        return QMM_ERR_ALIGN;
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return QMM_ERR_DEVICE;
    if (K == 0)
        return from_cuda(cudaMemsetAsync(y, 0, static_cast<size_t>(M) * N * 2, stream));
    DecodePlan plan;
    if (!decode_plan(M, N, K, group, bits, zeros != nullptr, true, f->num_sms, f->smem_pair, f->smem_optin, &plan))
        return QMM_ERR_UNSUPPORTED;
    DecodeParams d;
    std::memset(&d, 0, sizeof(d));
    d.x = static_cast<const uint16_t *>(x);
    d.packed = tiled;
    d.scales = static_cast<const uint16_t *>(scales);
    d.zeros = zeros;
    d.y = y;
    d.status = f->status;
    d.row_bytes = static_cast<long long>(K) * bits / 8;
    d.M = M;
    d.N = N;
    d.K = K;
    d.group_log2 = group == 64 ? 6 : 7;
    d.y_bf16 = y_dtype == QMM_BF16;
    d.x_bf16 = x_dtype == QMM_BF16;
    d.zero_const = zeros ? 0 : zero_const;
    d.vec_sz = aligned(scales, 16) && (!zeros || aligned(zeros, 8));
    d.pl = plan;
    return from_cuda(launch_decode(d, bits, true, stream));
}

qmm_status qmm_set_gemv_kernel(int kernel)
{
    if (kernel != QMM_GEMV_AUTO && kernel != QMM_GEMV_SKINNY)
        return QMM_ERR_SHAPE;
    g_gemv_kernel.store(kernel, std::memory_order_relaxed);
    return QMM_OK;
}

qmm_status qmm_gemm(const void *x, qmm_dtype x_dtype, const uint8_t *packed, int bits,
                    int group, const void *scales, const uint8_t *zeros, int zero_const,
                    void *y, qmm_dtype y_dtype, int M, int N, int K, cudaStream_t stream)
{
    qmm_status st = check_qmm_args(x, packed, bits, group, scales, zero_const, zeros, y, M, N, K);
    if (st != QMM_OK)
        return st;
    if (M != 0 && M < 17)
        return QMM_ERR_SHAPE;
    if (x_dtype != y_dtype || (x_dtype != QMM_F16 && x_dtype != QMM_BF16))
        return QMM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0)
        return QMM_OK;
    if (K > 0 && (!aligned(x, 16) || !aligned(packed, 16) || !aligned(y, 16) ||
                  (static_cast<long long>(K) * bits / 8) % 16))
        return QMM_ERR_ALIGN;
    if (K > 0 && !gemm_supports_bits(bits))
        return QMM_ERR_UNSUPPORTED;
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return QMM_ERR_DEVICE;
    if (K == 0)
        return from_cuda(cudaMemsetAsync(y, 0, static_cast<size_t>(M) * N * 2, stream));
    return gemm_dispatch(x, x_dtype == QMM_BF16, packed, bits, group, scales, zeros, zero_const,
                         y, M, N, K, f->status, f->num_sms, f->smem_optin, stream);
}

qmm_status qmm_w4a8(const int8_t *xq, const void *sa, const uint8_t *w4, const void *ws,
                    int group, void *y, int32_t *acc_out, int M, int N, int K,
                    cudaStream_t stream)
{
    if (M < 0 || N < 0 || K < 0)
        return QMM_ERR_SHAPE;
    if (group != 32 && group != 64 && group != 128)
        return QMM_ERR_SHAPE;
    if (K % group || M > 64)
        return QMM_ERR_SHAPE;
    if (M == 0 || N == 0)
        return QMM_OK;
    if (!y)
        return QMM_ERR_NULL;
    if (K > 0 && (!xq || !sa || !w4 || !ws))
        return QMM_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(w4, 16) || !aligned(ws, 2) || !aligned(sa, 2) ||
        !aligned(y, 2) || (acc_out && !aligned(acc_out, 4)))
        return QMM_ERR_ALIGN;
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return QMM_ERR_DEVICE;
    if (K == 0) {
        cudaError_t e = cudaMemsetAsync(y, 0, static_cast<size_t>(M) * N * 2, stream);
        return from_cuda(e);
    }
    return wxa8_dispatch(4, xq, sa, w4, ws, group, y, acc_out, M, N, K, f->status, f->num_sms,
                         f->smem_optin, f->smem_pair,
                         g_gemv_kernel.load(std::memory_order_relaxed) == QMM_GEMV_AUTO, stream);
}

qmm_status qmm_w8a8(const int8_t *xq, const void *sa, const int8_t *w8, const void *ws,
                    int group, void *y, int32_t *acc_out, int M, int N, int K,
                    cudaStream_t stream)
{
    if (M < 0 || N < 0 || K < 0)
        return QMM_ERR_SHAPE;
    if (group != 32 && group != 64 && group != 128)
        return QMM_ERR_SHAPE;
    if (K % group || M > 64)
        return QMM_ERR_SHAPE;
    if (M == 0 || N == 0)
        return QMM_OK;
    if (!y)
        return QMM_ERR_NULL;
    if (K > 0 && (!xq || !sa || !w8 || !ws))
        return QMM_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(w8, 16) || !aligned(ws, 2) || !aligned(sa, 2) ||
        !aligned(y, 2) || (acc_out && !aligned(acc_out, 4)))
        return QMM_ERR_ALIGN;
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return QMM_ERR_DEVICE;
    if (K == 0)
        return from_cuda(cudaMemsetAsync(y, 0, static_cast<size_t>(M) * N * 2, stream));
    return wxa8_dispatch(8, xq, sa, reinterpret_cast<const uint8_t *>(w8), ws, group, y, acc_out, M, N,
                         K, f->status, f->num_sms, f->smem_optin, f->smem_pair,
                         g_gemv_kernel.load(std::memory_order_relaxed) == QMM_GEMV_AUTO, stream);
}

qmm_status qmm_quantize_act(const void *x, int8_t *xq, void *sa, int M, int K, cudaStream_t stream)
{
    if (M < 0 || K < 0 || K % 8)
        return QMM_ERR_SHAPE;
    if (M == 0)
        return QMM_OK;
    if (!sa || (K > 0 && (!x || !xq)))
        return QMM_ERR_NULL;
    if (!aligned(sa, 2) || (K > 0 && (!aligned(x, 16) || !aligned(xq, 16))))
        return QMM_ERR_ALIGN;
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return QMM_ERR_DEVICE;
    if (K == 0)   // max over an empty row is 0: every scale is 0
        return from_cuda(cudaMemsetAsync(sa, 0, static_cast<size_t>(M) * 2, stream));
    return from_cuda(launch_quantize_act(static_cast<const uint16_t *>(x), xq, static_cast<uint16_t *>(sa),
                                         M, K, stream));
}

qmm_status qmm_kv_append(const qmm_paged_kv *kv, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                         const void *q, int64_t q_stride, void *q_out, int q_heads, const float *cos_sin, int rot,
                         int rope_len, int interleaved, cudaStream_t stream)
{
    const qmm_status st = check_paged(kv);
    if (st != QMM_OK)
        return st;
    if (rot < 0 || rot > kv->head_dim || rot % 16 || rope_len < 0 || q_heads < 0)
        return QMM_ERR_SHAPE;
    if (kv->tokens > 1 && (k_stride < 0 || v_stride < 0 || (q && q_stride < 0)))
        return QMM_ERR_SHAPE;
    if (kv->tokens > 1 && (k_stride % 8 || v_stride % 8 || (q && q_stride % 8)))
        return QMM_ERR_ALIGN;
    if (kv->batch == 0 || kv->tokens == 0)
        return QMM_OK;
    if (!k || !v || (rot > 0 && !cos_sin) || !q != !q_out)
        return QMM_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16) || !aligned(cos_sin, 16))
        return QMM_ERR_ALIGN;
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return QMM_ERR_DEVICE;
    AppendParams p;
    std::memset(&p, 0, sizeof(p));
    p.kv = *kv;
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q = static_cast<const uint16_t *>(q);
    p.q_out = static_cast<uint16_t *>(q_out);
    p.cos_sin = cos_sin;
    p.status = f->status;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_stride = q_stride;
    p.q_heads = q ? q_heads : 0;
    p.rot = rot;
    p.rope_len = rope_len;
    p.interleaved = interleaved != 0;
    p.by_page = fast_div(kv->page_size);
    return from_cuda(launch_kv_append(p, stream));
}

size_t qmm_paged_attn_workspace(int q_heads, int kv_heads, int head_dim, int max_q)
{
    if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads || (head_dim != 64 && head_dim != 128) || max_q < 0)
        return 0;
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return 0;
    return attn_workspace_bytes(q_heads, kv_heads, head_dim, max_q, f->num_sms);
}

qmm_status qmm_paged_attn(const qmm_paged_kv *kv, const void *q, int64_t q_stride, int q_heads, float scale,
                          int causal, int window, void *out, float *lse, int max_q, int max_kv, void *workspace,
                          size_t workspace_bytes, cudaStream_t stream)
{
    const qmm_status st = check_paged(kv);
    if (st != QMM_OK)
        return st;
    if (q_heads < 1 || q_heads % kv->kv_heads || window < 0 || (window > 0 && !causal) || max_q < 0 || max_kv < 0 ||
        !(scale > 0.f) || !(scale <= 2.0e38f) || (kv->tokens > 1 && q_stride < 0))   // scale log2(e) is finite
        return QMM_ERR_SHAPE;
    if (kv->tokens > 1 && q_stride % 8)
        return QMM_ERR_ALIGN;
    if (kv->batch == 0 || kv->tokens == 0)
        return QMM_OK;
    if (!q || !out || !workspace)
        return QMM_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(lse, 4))
        return QMM_ERR_ALIGN;
    // row tiles of the batch are counted in 32 bits (no sequence has more than `tokens`)
    const int group = q_heads / kv->kv_heads;
    if ((static_cast<long long>(std::min(max_q, kv->tokens)) * group / 16 + 1) * kv->batch > 0x7fffffffLL ||
        static_cast<long long>(kv->tokens) * group > 0x7fffffffLL)
        return QMM_ERR_UNSUPPORTED;
    // max_q = 0 says that no sequence has a token, so that there is nothing to do; that is for
    // the device to check, where there is one, as for every other bound: one token is
    // answered, more are recorded
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return max_q == 0 ? QMM_OK : QMM_ERR_DEVICE;
    if (workspace_bytes < attn_workspace_bytes(q_heads, kv->kv_heads, kv->head_dim, max_q, f->num_sms))
        return QMM_ERR_SHAPE;
    AttnParams p;
    std::memset(&p, 0, sizeof(p));
    p.kv = *kv;
    p.q = static_cast<const uint16_t *>(q);
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.status = f->status;
    p.q_stride = q_stride;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.q_heads = q_heads;
    p.group = group;
    p.causal = causal != 0;
    p.window = window;
    return from_cuda(attn_dispatch(p, max_q, max_kv, workspace, f->num_sms, stream));
}

qmm_status qmm_kv4_append(const qmm_paged_kv4 *kv, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                          const void *q, int64_t q_stride, void *q_out, int q_heads, const float *cos_sin, int rot,
                          int rope_len, int interleaved, const void *q_norm, const void *k_norm, float eps,
                          cudaStream_t stream)
{
    Kv4AppendParams p;
    std::memset(&p, 0, sizeof(p));
    const qmm_status st = check_kv4(kv, &p.kv, &p.sc);
    if (st != QMM_OK)
        return st;
    if (rot < 0 || rot > kv->head_dim || rot % 16 || rope_len < 0 || q_heads < 0 || !(eps >= 0.f) || !(eps < INFINITY))
        return QMM_ERR_SHAPE;
    if (q_heads > 65536)
        return QMM_ERR_UNSUPPORTED;
    if (kv->tokens > 1 && (k_stride < 0 || v_stride < 0 || (q && q_stride < 0)))
        return QMM_ERR_SHAPE;
    if (kv->tokens > 1 && (k_stride % 8 || v_stride % 8 || (q && q_stride % 8)))
        return QMM_ERR_ALIGN;
    if (kv->batch == 0 || kv->tokens == 0)
        return QMM_OK;
    if (!k || !v || (rot > 0 && !cos_sin) || !q != !q_out)
        return QMM_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16) || !aligned(cos_sin, 16) ||
        !aligned(q_norm, 16) || !aligned(k_norm, 16))
        return QMM_ERR_ALIGN;
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return QMM_ERR_DEVICE;
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q = static_cast<const uint16_t *>(q);
    p.q_out = static_cast<uint16_t *>(q_out);
    p.cos_sin = cos_sin;
    p.status = f->status;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_stride = q_stride;
    p.q_heads = q ? q_heads : 0;
    p.rot = rot;
    p.rope_len = rope_len;
    p.interleaved = interleaved != 0;
    p.by_page = fast_div(kv->page_size);
    p.q_norm = static_cast<const uint16_t *>(q_norm);
    p.k_norm = static_cast<const uint16_t *>(k_norm);
    p.eps = eps;
    p.one = 1.f;
    return from_cuda(launch_kv4_append(p, stream));
}

qmm_status qmm_kv4_read(const qmm_paged_kv4 *kv, void *k_out, void *v_out, cudaStream_t stream)
{
    Kv4ReadParams p;
    std::memset(&p, 0, sizeof(p));
    const qmm_status st = check_kv4(kv, &p.kv, &p.sc);
    if (st != QMM_OK)
        return st;
    if (kv->batch == 0 || kv->tokens == 0)
        return QMM_OK;
    if (!k_out || !v_out)
        return QMM_ERR_NULL;
    if (!aligned(k_out, 16) || !aligned(v_out, 16))
        return QMM_ERR_ALIGN;
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return QMM_ERR_DEVICE;
    p.k = static_cast<uint16_t *>(k_out);
    p.v = static_cast<uint16_t *>(v_out);
    p.status = f->status;
    p.by_page = fast_div(kv->page_size);
    p.by_heads = fast_div(kv->kv_heads);
    return from_cuda(launch_kv4_read(p, f->num_sms, stream));
}

size_t qmm_kv4_attn_workspace(int q_heads, int kv_heads, int head_dim, int max_q)
{
    if (q_heads < 1 || kv_heads < 1 || q_heads > 65536 || q_heads % kv_heads || (head_dim != 64 && head_dim != 128) || max_q < 0)
        return 0;
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return 0;
    return kv4_attn_workspace_bytes(q_heads, kv_heads, head_dim, max_q, f->num_sms);
}

size_t qmm_kv4_attn_more_workspace(int batch, int tokens, int q_heads, int kv_heads, int head_dim, int max_q, int max_kv,
                                   int sinks)
{
    if (batch < 1 || tokens < 1 || sinks < 0 || max_kv < 0 || qmm_kv4_attn_workspace(q_heads, kv_heads, head_dim, max_q) == 0)
        return 0;
    return kv4_attn_unpack_bytes(batch, tokens, q_heads / kv_heads, kv_heads, head_dim, max_q, max_kv, sinks);
}

qmm_status qmm_kv4_attn(const qmm_paged_kv4 *kv, const void *q, int64_t q_stride, int q_heads, float scale, int causal,
                        int window, int sinks, void *out, float *lse, int max_q, int max_kv, void *workspace,
                        size_t workspace_bytes, cudaStream_t stream)
{
    Kv4AttnParams p;
    std::memset(&p, 0, sizeof(p));
    const qmm_status st = check_kv4(kv, &p.kv, &p.sc);
    if (st != QMM_OK)
        return st;
    if (q_heads < 1 || q_heads % kv->kv_heads || window < 0 || (window > 0 && !causal) || sinks < 0 ||
        (sinks > 0 && window == 0) || max_q < 0 || max_kv < 0 || !(scale > 0.f) || !(scale <= 2.0e38f) ||
        (kv->tokens > 1 && q_stride < 0))   // scale log2(e) is finite
        return QMM_ERR_SHAPE;
    if (q_heads > 65536)
        return QMM_ERR_UNSUPPORTED;
    if (kv->tokens > 1 && q_stride % 8)
        return QMM_ERR_ALIGN;
    if (kv->batch == 0 || kv->tokens == 0)
        return QMM_OK;
    if (!q || !out || !workspace)
        return QMM_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(lse, 4))
        return QMM_ERR_ALIGN;
    if (!kv4_set_units(p))
        return QMM_ERR_UNSUPPORTED;
    // row tiles of the batch are counted in 32 bits (no sequence has more than `tokens`)
    const int group = q_heads / kv->kv_heads;
    if ((static_cast<long long>(std::min(max_q, kv->tokens)) * group / 8 + 1) * kv->batch > 0x7fffffffLL ||
        static_cast<long long>(kv->tokens) * group > 0x7fffffffLL)
        return QMM_ERR_UNSUPPORTED;
    // (max_q = 0: as for qmm_paged_attn)
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return max_q == 0 ? QMM_OK : QMM_ERR_DEVICE;
    const size_t need = kv4_attn_workspace_bytes(q_heads, kv->kv_heads, kv->head_dim, max_q, f->num_sms);
    if (workspace_bytes < need)
        return QMM_ERR_SHAPE;
    // (tensor copies read the converted keys from multiples of 128 bytes of the scratch)
    const size_t more = aligned(workspace, 128) ? workspace_bytes - need : 0;
    p.q = static_cast<const uint16_t *>(q);
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.status = f->status;
    p.q_stride = q_stride;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.q_heads = q_heads;
    p.group = group;
    p.causal = causal != 0;
    p.window = window;
    p.sinks = sinks;
    return from_cuda(kv4_attn_dispatch(p, max_q, max_kv, workspace, more, f->num_sms, stream));
}

qmm_status qmm_watchdog_selftest(cudaStream_t stream)
{
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return QMM_ERR_DEVICE;
    watchdog_selftest_kernel<<<1, 32, 0, stream>>>(f->status);
    return from_cuda(cudaGetLastError());
}

qmm_status qmm_device_status(cudaStream_t stream)
{
    const DeviceFacts *f = device_facts();
    if (!f || f->usable != QMM_OK)
        return QMM_ERR_DEVICE;
    if (cudaStreamSynchronize(stream) != cudaSuccess) {
        cudaGetLastError();
        return QMM_ERR_CUDA;
    }
    int v = 0;
    if (cudaMemcpy(&v, f->status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess)
        return QMM_ERR_CUDA;
    if (v != 0) {
        const int zero = 0;
        cudaMemcpy(f->status, &zero, sizeof(int), cudaMemcpyHostToDevice);
    }
    return static_cast<qmm_status>(v);
}

}  // extern "C"
