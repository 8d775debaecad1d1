// paged.cuh -- device helpers of the paged key / value cache kernels: places in
// the cache, asynchronous 16-byte copies, 16-bit conversions, and the split of an
// attention call's work over the blocks.
#pragma once

#include "common.cuh"
#include "paged.h"

namespace qmm {

namespace {

// ---- small numeric helpers ------------------------------------------------------
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// fp32 -> two 16-bit values (lo = a), round to nearest even
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float a, float b)
{
    uint32_t d;
    if constexpr (BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
}

template <bool BF16>
__device__ __forceinline__ float lo16(uint32_t w)
{
    return BF16 ? __uint_as_float(w << 16) : f16_bits_to_f32(static_cast<uint16_t>(w));
}

template <bool BF16>
__device__ __forceinline__ float hi16(uint32_t w)
{
    return BF16 ? __uint_as_float(w & 0xFFFF0000u) : f16_bits_to_f32(static_cast<uint16_t>(w >> 16));
}

// ---- the end of a row -------------------------------------------------------------
// A row's maximum m (in powers of two), its sum l of 2^(s - m + shift) and what they give.
// l is zero only where the row sees no key (the largest weight is 2^-8 at least): its output
// is zero and its log sum -infinity.  NaN and infinite scores leave NaN in l, and so in both.
__device__ __forceinline__ float row_inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }

template <bool BF16>
__device__ __forceinline__ float row_log_sum(float m, float l)
{
    constexpr float kShift = BF16 ? 0.f : 7.f;
    return l == 0.f ? -INFINITY : (m - kShift + log2f(l)) * 0.6931471805599453f;
}

// ---- asynchronous copies --------------------------------------------------------
// 16 bytes global -> shared through L2; with ok == false 16 zero bytes (nothing is
// read, `src` only has to be a valid address).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool ok)
{
    const int n = ok ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_async_wait_group()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---- the batch ----------------------------------------------------------------------
// The new tokens of sequence b: first token and count, held to 0 .. tokens.
__device__ __forceinline__ int2 seq_tokens(const qmm_paged_kv &kv, int b)
{
    const int t0 = min(max(kv.cu_q[b], 0), kv.tokens);
    const int t1 = min(max(kv.cu_q[b + 1], t0), kv.tokens);
    return make_int2(t0, t1 - t0);
}

// Keys of a sequence at most: the kernels look up to a few thousand keys past a sequence's
// end (whole tiles, those loaded ahead) before they see that nothing is there.
constexpr int kMostKeys = 0x7fffffff - 16383;

// What a sequence's row of the block table can hold.
__device__ __forceinline__ int table_keys(const qmm_paged_kv &kv)
{
    return static_cast<int>(min(static_cast<long long>(kv.blocks) * kv.page_size, static_cast<long long>(kMostKeys)));
}

// A sequence's number of keys, held to that.
__device__ __forceinline__ int seq_keys(const qmm_paged_kv &kv, int n, int *status)
{
    const int most = table_keys(kv);
    if (n > most) {
        record_error(status, QMM_ERR_INDEX);
        return most;
    }
    return max(n, 0);
}

// Element offset of (sequence b, key, head 0) in the cache, or -1 (recorded) for a
// page number out of range.  key is in [0, blocks * page_size).
__device__ __forceinline__ long long key_offset(const qmm_paged_kv &kv, const FastDiv &by_page, int b, int key,
                                                int *status)
{
    const int blk = by_page(key);
    const int slot = key - blk * kv.page_size;
    const int page = kv.block_table[static_cast<long long>(b) * kv.blocks + blk];
    if (page < 0 || page >= kv.num_pages) {
        record_error(status, QMM_ERR_INDEX);
        return -1;
    }
    return page * kv.page_stride + slot * kv.slot_stride;
}

// The sequence that owns token t (the number of sequences that end at or before
// t), its end cu_q[b + 1] and its key count, by one warp: lanes look at 32
// sequences at a time.  b = batch if no sequence owns it.
__device__ __forceinline__ void find_sequence(const qmm_paged_kv &kv, int t, int lane, int &b, int &end, int &keys)
{
    for (int b0 = 0; b0 < kv.batch; b0 += 32) {
        const int i = b0 + lane;
        int e = 0x7fffffff, k = 0;
        if (i < kv.batch) {
            e = kv.cu_q[i + 1];
            k = kv.kv_len[i];
        }
        const int cnt = __popc(__ballot_sync(0xffffffffu, e <= t));
        if (cnt < 32) {
            b = b0 + cnt;
            end = __shfl_sync(0xffffffffu, e, cnt);
            keys = __shfl_sync(0xffffffffu, k, cnt);
            return;
        }
    }
    b = kv.batch;
}

// ---- the split of an attention call --------------------------------------------------
// An item is one row tile of one sequence with one key head: tile_rows consecutive rows
// of the sequence's (token, query head of the key head) pairs, token-major, with the
// keys [lo, hi) that any of them sees.  Its work is counted in units of KEYS keys
// (aligned to KEYS), at least one so that rows without keys are written too.
struct RowTile {
    int b;          // sequence
    int t0;         // its first new token
    int n;          // its new tokens
    int row0;       // first row of the tile
    int rows;       // rows in the tile (0: the tile does not exist)
    int kv;         // keys of the sequence
    int lo, hi;     // keys some row of the tile sees (SINKS: see row_tile)
    int unit0, units;
};

// First key that a row at position pos sees under a window (> 0).  Compared before the
// difference is taken: pos may be negative (padding) and the window as large as an int.
__host__ __device__ __forceinline__ int window_start(int pos, int window) { return pos >= window ? pos - window + 1 : 0; }

// With first tokens that stay visible (SINKS, p.sinks) an item's keys are numbered along an
// axis without the hidden ones between those and the window: places 0 .. hi, which the units
// count along, place i being key i + (i < p.sinks ? 0 : lo).  Every row of a tile that has such
// a gap sees the first tokens (its position lies past the window's start).
template <int KEYS, bool SINKS = false>
__device__ __forceinline__ RowTile row_tile(const AttnParams &p, int i)
{
    RowTile r;
    r.b = p.by_tiles(i);
    r.row0 = (i - r.b * p.row_tiles) * p.tile_rows;
    const int keys = p.kv.kv_len[r.b];   // (the lengths' loads are under way together)
    const int2 tn = seq_tokens(p.kv, r.b);
    r.t0 = tn.x;
    r.n = tn.y;
    const long long all = static_cast<long long>(r.n) * p.group;
    r.rows = static_cast<int>(min(static_cast<long long>(p.tile_rows), max(0LL, all - r.row0)));
    r.kv = seq_keys(p.kv, keys, p.status);
    r.lo = r.hi = r.unit0 = r.units = 0;
    if (r.rows == 0)
        return r;
    const int first = r.kv - r.n + p.by_group(r.row0);                     // position of the first row
    const int last = r.kv - r.n + p.by_group(r.row0 + r.rows - 1);
    r.hi = p.causal ? min(r.kv, max(0, last + 1)) : r.kv;
    r.lo = p.window > 0 ? min(r.hi, window_start(first, p.window)) : 0;
    if constexpr (SINKS) {
        r.lo = max(0, r.lo - p.sinks);
        r.hi -= r.lo;
        r.units = max(1, (r.hi + KEYS - 1) / KEYS);
        return r;
    }
    r.unit0 = r.lo / KEYS;
    r.units = max(1, (r.hi + KEYS - 1) / KEYS - r.unit0);
    return r;
}

// Visible keys [jmin, jmax] of row `row` (of the whole sequence) in the tile's
// sequence; an empty range for rows past the tile.
__device__ __forceinline__ int2 row_keys(const AttnParams &p, const RowTile &r, int row)
{
    if (row >= r.row0 + r.rows)
        return make_int2(0, -1);
    const int pos = r.kv - r.n + p.by_group(row);
    return make_int2(p.window > 0 ? window_start(pos, p.window) : 0, p.causal ? min(r.kv - 1, pos) : r.kv - 1);
}

// The same in places (SINKS).
__device__ __forceinline__ int2 row_places(const AttnParams &p, const RowTile &r, int row)
{
    const int2 k = row_keys(p, r, row);
    return make_int2(k.x - r.lo, k.y - r.lo);
}

// Where a block's share of the work starts.  All items of the call lie on one
// line, row tiles in order, key heads within a row tile; an item is SETUP + units
// long (SETUP: what starting and finishing an item costs, in units; its first unit
// lies SETUP behind its start).  Block c takes the stretch [c * chunk, (c + 1) *
// chunk), chunk = max(min_chunk, total / grid rounded up), so every block has the
// same work however ragged the batch is.  An item that crosses a block's border
// leaves partial results (at most two per block) that a second kernel joins (attn.cu).
// The split depends on the lengths alone, so results are the same run to run.  With
// p.unsplit a block takes the items that start in its stretch, whole.
struct Share {
    long long at, end;       // the block's stretch
    long long chunk;
    long long start;         // where the item (i, h) that holds `at` starts
    int i, h;                // row tile and key head of it
    RowTile r;               // the row tile
};

// a / b for a >= 0, b > 0.  The line is nearly always shorter than 2^31, and a 64-bit
// division is some 600 cycles on a path that every block waits for.
__device__ __forceinline__ long long divide(long long a, long long b)
{
    return ((a | b) >> 31) == 0 ? static_cast<long long>(static_cast<unsigned>(a) / static_cast<unsigned>(b)) : a / b;
}

// Called by all THREADS threads of the block; `red` is scratch of THREADS / 32
// words of 8 bytes, `out` the shared result.
template <int KEYS, int SETUP, int THREADS, bool SINKS = false>
__device__ __forceinline__ void find_share(const AttnParams &p, long long *red, Share *out)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (p.whole && !p.unsplit) {   // cluster (or block) c holds item c
        if (tid == 0) {
            const int item = blockIdx.x / p.cluster, i = item / p.kv.kv_heads;
            const RowTile r = row_tile<KEYS, SINKS>(p, i);
            out->i = i;
            out->r = r;
            out->h = item - i * p.kv.kv_heads;
            out->at = out->start = 0;
            out->end = r.units ? SETUP + r.units : 0;
            out->chunk = 1LL << 40;
            if (r.row0 == 0 && static_cast<long long>(r.n) * p.group > static_cast<long long>(p.row_tiles) * p.tile_rows)
                record_error(p.status, QMM_ERR_INDEX);
        }
        __syncthreads();
        return;
    }
    const int tiles = p.kv.batch * p.row_tiles;
    const int per = (tiles + THREADS - 1) / THREADS;
    const int i0 = min(tiles, tid * per), i1 = min(tiles, i0 + per);
    long long sum = 0;
    RowTile r;
    for (int i = i0; i < i1; ++i) {
        r = row_tile<KEYS, SINKS>(p, i);
        sum += static_cast<long long>(r.units ? SETUP + r.units : 0) * p.kv.kv_heads;
        if (r.row0 == 0 && static_cast<long long>(r.n) * p.group > static_cast<long long>(p.row_tiles) * p.tile_rows)
            record_error(p.status, QMM_ERR_INDEX);   // more new tokens than max_q
    }
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += v;
    }
    if (lane == 31)
        red[warp] = incl;
    if (tid == 0)
        out->at = out->end = out->start = 0;
    __syncthreads();
    long long base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        const long long v = red[w];
        if (w < warp)
            base += v;
        total += v;
    }
    const long long before = base + incl - sum;
    const long long chunk = max(static_cast<long long>(p.min_chunk), divide(total + gridDim.x - 1, gridDim.x));
    const long long at = chunk * blockIdx.x;
    if (tid == 0)
        out->chunk = chunk;
    if (at < total && before <= at && at < before + sum) {
        long long start = before;
        for (int i = i0; i < i1; ++i) {
            if (per > 1)
                r = row_tile<KEYS, SINKS>(p, i);
            const int len = r.units ? SETUP + r.units : 0;
            const long long all = static_cast<long long>(len) * p.kv.kv_heads;
            if (at < start + all) {
                out->i = i;
                out->r = r;
                out->h = static_cast<int>(divide(at - start, len));
                out->start = start + static_cast<long long>(out->h) * len;
                out->at = at;
                out->end = min(total, at + chunk);
                break;
            }
            start += all;
        }
    }
    __syncthreads();
}

// One segment of a block's share: `units` >= 1 units from unit `off` of an item (row
// tile r, head h) that starts at `start` of the line.
struct Segment {
    RowTile r;
    int h, off, units;
    long long start;
};

// Walks a share.  next() gives its segments in order.
template <int KEYS, int SETUP, bool SINKS = false>
struct Walk {
    long long at, end, chunk, start;
    int i, h;
    RowTile r;
    __device__ __forceinline__ void begin(const Share &s)
    {
        at = s.at;
        end = s.end;
        chunk = s.chunk;
        start = s.start;
        i = s.i;
        h = s.h;
        r = s.r;
    }
    // on to the next item, which starts len further on
    __device__ __forceinline__ bool advance(const AttnParams &p, int len)
    {
        start += len;
        if (++h == p.kv.kv_heads) {
            h = 0;
            do {
                if (++i >= p.kv.batch * p.row_tiles)
                    return false;
                r = row_tile<KEYS, SINKS>(p, i);
            } while (r.units == 0);
        }
        return true;
    }
    __device__ __forceinline__ bool next(const AttnParams &p, Segment &s)
    {
        if (p.unsplit) {
            while (at < end && start < at)       // began in an earlier block
                if (!advance(p, SETUP + r.units))
                    at = end;
            if (at >= end || start >= end)
                return false;
            s.r = r;
            s.h = h;
            s.off = 0;
            s.units = r.units;
            s.start = start;
            if (!advance(p, SETUP + r.units))
                at = end;                        // that was the last item
            return true;
        }
        while (at < end) {
            const int len = SETUP + r.units;
            if (at >= start + len) {
                if (!advance(p, len))
                    return false;   // not reached: the stretch ahead belongs to some tile
                continue;
            }
            const long long to = min(end, start + len);
            const int a = max(0, static_cast<int>(at - start) - SETUP), b = static_cast<int>(to - start) - SETUP;
            at = to;
            if (b <= a)
                continue;              // only the item's start-up lies here
            s.r = r;
            s.h = h;
            s.off = a;
            s.units = b - a;
            s.start = start;
            return true;
        }
        return false;
    }
};

// Partial-result slot of a segment of block c: 1 where the item begins in c, else 0.
__device__ __forceinline__ int part_slot(const Segment &s) { return 2 * static_cast<int>(blockIdx.x) + (s.off == 0 ? 1 : 0); }
__device__ __forceinline__ bool is_whole(const Segment &s) { return s.units == s.r.units; }
// Whether this block holds the last part, but not all, of the item.
__device__ __forceinline__ bool is_last_part(const Segment &s) { return s.off > 0 && s.off + s.units == s.r.units; }

// What the joining kernel needs of an item: its first block (the one that holds its
// first unit), its rows, first row and token, and its key head.
template <int SETUP>
__device__ __forceinline__ void write_meta(const AttnParams &p, const Segment &s, long long chunk)
{
    p.meta[2 * blockIdx.x] = make_int4(static_cast<int>(divide(s.start + SETUP, chunk)), s.r.rows, s.r.row0, s.r.t0);
    p.meta[2 * blockIdx.x + 1] = make_int4(s.h, 0, 0, 0);
}

}  // namespace

}  // namespace qmm
