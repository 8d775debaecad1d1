// kv4_attn.cu -- qmm_kv4_attn: kernel choice and split sizes.
#include <algorithm>

#include "kv4.h"
#include "paged.cuh"

namespace qmm {

namespace {

// Blocks that a split goes over: of four warps of the kernel for few rows, or one per SM.
int grid_of(bool few, int rows, int num_sms) { return few ? kv4_blocks_per_sm(rows, 4) * num_sms : num_sms; }

// Work a block takes at least, in units: below this a split costs more (a second kernel,
// the partial results) than the longer walk.
constexpr int kMinUnits = 3, kMinChunkUnits = 4;

// Few rows, whole items in clusters against a split over all blocks: a cluster's block walks
// units / c, a split one units * items / blocks and the joining kernel's time, some
// kJoinUnits; and not more than kMostUnits, since whole items are not balanced where
// lengths differ.  One token over 4000 keys of 8 heads 7.6 us in clusters of 8 (4: 9.9, 1:
// 24.6, split 11.1); 16 over 2000 15.1 in 2 (split 19.3), 32 over 4000 40.4 in 1 (42.5).
constexpr int kJoinUnits = 4, kMostUnits = 10;

// Few rows, whole items in blocks of four warps, more of them than run at once: blocks start as
// others end, without a joining kernel and with fewer items cut in two; at the end the
// last ones run alone, which costs the more the longer the items and the fewer they are.  Up
// to kWholeUnits units and kMoreUnits for each time that the blocks are filled: 512 items of 700
// keys 19.1 us (split 24.3), of 140 .. 1400 27.0 (27.0), of 280 .. 2800 49.2 (41.6); 2048 of
// 1400 95.4 (105.9), of 280 .. 2800 115.5 (117.2), of 560 .. 5600 223 (213).
constexpr int kWholeUnits = 6, kMoreUnits = 5;

// Many rows: work of the longest item (setup and units) up to which blocks take whole items,
// and the same where every item has a block of its own (as attn.cu).
constexpr int kUnsplitWork = 12, kWholeWork = 10;

// Rows (token, query head) per key head of the kernel for few rows: two column tiles of the
// matrix instructions.  More go to it, sixteen at a time, where these items all run at once in
// clusters (128 rows over 2000 keys 13.1 us, many-row kernel 16.3; but 32 over 2000 of 64
// sequences 110 and 103).
constexpr int kFewRows = 16;

// Where keys are converted once, into scratch, and read by the 16-bit form of the kernel for many
// rows, in place of by every row tile that sees them: it costs a launch and a pass over the keys,
// and saves some of each tile's time per key.  So from so many row tiles, and so much work, tiles
// x keys over all heads and sequences, on (us, by every tile and once, for heads of 64 and of 128; in a
// graph, codes at random; called one by one the launch costs some 2 us more):
//   heads  new  keys    tiles  work      64: every  once     128: every  once
//   64/8   128  16384   4      2^19      50.9       50.8     69.8        69.6
//   64/8   256  16384   8      2^20      86.5       78.4     119.3       105.9
//   8/8    2048 8192    8      2^19      46.4       44.3     64.8        58.7
//   8/8    2048 16384   8      2^20      82.9       76.0     113.9       101.5
//   64/8   1024 1024    32     2^18      32.3       29.5     42.0        37.0
//   32/8   1024 4096    16     2^19      49.2       44.8     68.5        59.3
//   32/8   2048 2048    32     2^19      37.9       34.8     54.9        47.2
//   8/1    2048 2048    64     2^17      20.1       20.1     25.0        25.5
//   8/1    1024 16384   32     2^19      48.1       46.0     61.3        59.2
//   64/8   2048 16384   64     2^23      558        452      786         587
constexpr int kUnpackTiles = 8;
constexpr long long kUnpackWork = 1LL << 19;
// Bytes of converted keys at most.
constexpr long long kUnpackMost = 1LL << 30;

// (Row tiles per sequence on average: a prompt beside many sequences of a token each would have
// all their keys converted for few rows.  keys: what a row tile sees at most.)
bool unpack_pays(int batch, int tokens, int group, int kv_heads, int max_q, long long keys)
{
    const double rows = 2 * chunk_stream_rows(group);
    const double tiles = std::min(static_cast<double>(max_q), static_cast<double>(tokens) / batch) * group / rows;
    return tiles > kUnpackTiles - 1 && tiles * static_cast<double>(keys) * kv_heads * batch >= kUnpackWork;
}

// Places per sequence of the converted keys.
long long unpack_cap(long long max_kv) { return (max_kv + 127) / 128 * 128; }

// The block table of the converted keys, a page per sequence, before them.
size_t table_bytes(int batch) { return (static_cast<size_t>(batch) * 4 + 127) / 128 * 128; }

// Blocks of eight warps per item where every item gets a cluster (or block) of its own:
// clusters of the largest size that all run at once; 0: there are none.
int cluster_of(const Kv4AttnParams &p, int rows, long long items, long long span, int num_sms)
{
    const int keys = kv4_keys(p.kv.head_dim, 8), blocks = kv4_blocks_per_sm(rows, 8) * num_sms;
    const long long units = (span + keys - 1) / keys;
    for (int c = kMaxCluster; c >= 1; c /= 2)
        if (items * c <= blocks && (c == 1 || c / 2 < units) && (units + c - 1) / c <= kMostUnits &&
            (units + c - 1) / c <= items * units / blocks + kJoinUnits &&
            (c == 1 || items <= kv4_decode_clusters(p.kv.head_dim, p.kv.dtype == QMM_BF16, rows, c)))
            return c;
    return 0;
}

size_t scratch_bytes(bool few, int head_dim, int num_sms)
{
    const size_t g = grid_of(few, 8, num_sms), rows = few ? kDecodeRows : kChunkRows;
    return g * 32 + 2 * g * rows * (head_dim + 2) * 4;
}

// (a multiple of 16 bytes; the converted keys follow from a multiple of 128)
size_t scratch_bytes_most(int head_dim, int num_sms)
{
    return (std::max(scratch_bytes(true, head_dim, num_sms), scratch_bytes(false, head_dim, num_sms)) + 127) / 128 * 128;
}

}  // namespace

bool kv4_set_units(Kv4AttnParams &p)
{
    const unsigned long long page = p.kv.num_pages > 1 ? p.kv.page_stride : 0, slot = p.kv.page_size > 1 ? p.kv.slot_stride : 0;
    unsigned long long unit = 16;
    while (unit < 1u << 20 && (page | slot) % (2 * unit) == 0)
        unit *= 2;
    p.unit = static_cast<uint32_t>(unit);
    p.page_units = static_cast<uint32_t>(page / unit);
    p.slot_units = static_cast<uint32_t>(slot / unit);
    // (the last place is kept for "none")
    return (std::max(0, p.kv.num_pages - 1) * page + (p.kv.page_size - 1) * slot) / unit < 0xffffffffull;
}

size_t kv4_attn_workspace_bytes(int, int, int head_dim, int, int num_sms)
{
    return scratch_bytes_most(head_dim, num_sms);
}

size_t kv4_attn_unpack_bytes(int batch, int tokens, int group, int kv_heads, int head_dim, int max_q, long long max_kv, int sinks)
{
    if (sinks > 0 || max_kv <= 0 || max_kv > 0x7fffff00LL || group > 128 || batch > 65535 ||
        !unpack_pays(batch, tokens, group, kv_heads, max_q, max_kv))
        return 0;
    const double bytes = 4.0 * unpack_cap(max_kv) * kv_heads * head_dim * batch;
    return bytes > kUnpackMost ? 0 : table_bytes(batch) + static_cast<size_t>(bytes);
}

cudaError_t kv4_attn_dispatch(Kv4AttnParams &p, int max_q, long long max_kv, void *workspace, size_t more, int num_sms,
                              cudaStream_t stream)
{
    // no sequence has more tokens than the batch: a caller's large bound adds no row tiles
    max_q = std::max(1, std::min(max_q, p.kv.tokens));
    const long long most = static_cast<long long>(p.kv.blocks) * p.kv.page_size, q_rows = static_cast<long long>(max_q) * p.group;
    if (max_kv <= 0 || max_kv > most)
        max_kv = most;
    if (p.window >= most)   // no position lies further back
        p.window = 0;
    if (p.window == 0)
        p.sinks = 0;
    // keys of an item at most: a window's, the first tokens, and those its tokens see beyond each other
    const auto span_of = [&](int rows) {
        return p.window > 0 ? std::min(max_kv, static_cast<long long>(p.window) + p.sinks + rows / p.group + 1) : max_kv;
    };
    const int few_rows = q_rows <= 8 ? 8 : 16;
    const long long few_items = p.kv.batch * ((q_rows + few_rows - 1) / few_rows) * p.kv.kv_heads;
    const int cluster = cluster_of(p, few_rows, few_items, span_of(few_rows), num_sms);
    // (and queries that the other kernel's tensor copies do not take)
    const bool few = q_rows <= kFewRows || cluster > 0 || !attn_set_q_tma(p);
    p.tile_rows = few ? few_rows : 2 * chunk_stream_rows(p.group);
    p.row_tiles = static_cast<int>((q_rows + p.tile_rows - 1) / p.tile_rows);
    p.by_group = fast_div(p.group);
    p.by_tiles = fast_div(p.row_tiles);
    p.by_page = fast_div(p.kv.page_size);
    p.min_chunk = few ? kMinUnits : kMinChunkUnits;
    const long long items = static_cast<long long>(p.kv.batch) * p.row_tiles * p.kv.kv_heads, span = span_of(p.tile_rows);
    p.cluster = few && cluster > 0 ? cluster : 1;
    p.warps = few && cluster > 0 ? 8 : 4;
    const int keys = few ? kv4_keys(p.kv.head_dim, p.warps) : kChunkKeys, setup = few ? kDecodeSetup : kChunkSetup;
    const long long longest = (span + keys - 1) / keys;
    int grid = grid_of(few, p.tile_rows, num_sms);
    p.whole = few ? cluster > 0 || (longest <= kWholeUnits + kMoreUnits * items / grid && items <= 0x7fffffff)
                  : items <= grid ? longest + setup <= kWholeWork : longest + setup <= kUnsplitWork;
    p.unsplit = !few && p.whole && items > grid;
    if (p.whole && !p.unsplit)
        grid = static_cast<int>(items) * p.cluster;
    else if (p.unsplit)
        p.min_chunk = 1;
    else if (items * (longest + setup) < static_cast<long long>(grid) * p.min_chunk)
        grid = static_cast<int>((items * (longest + setup) + p.min_chunk - 1) / p.min_chunk);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const size_t g = grid_of(few, 8, num_sms);
    p.meta = reinterpret_cast<int4 *>(ws);
    p.part_ml = reinterpret_cast<float *>(ws + g * 32);
    p.part_o = p.part_ml + 2 * g * (few ? kDecodeRows : kChunkRows) * 2;
    const size_t unpack = few ? 0 : kv4_attn_unpack_bytes(p.kv.batch, p.kv.tokens, p.group, p.kv.kv_heads, p.kv.head_dim,
                                                              max_q, max_kv, p.sinks);
    if (unpack > 0 && unpack <= more && unpack_pays(p.kv.batch, p.kv.tokens, p.group, p.kv.kv_heads, max_q, span)) {
        Kv4ReadParams u = {};
        u.kv = p.kv;
        u.sc = p.sc;
        u.status = p.status;
        u.by_page = p.by_page;
        u.by_heads = fast_div(p.kv.kv_heads);
        u.cap = static_cast<int>(unpack_cap(max_kv));
        u.window = p.window;
        u.table = reinterpret_cast<int32_t *>(ws + scratch_bytes_most(p.kv.head_dim, num_sms));
        u.k = reinterpret_cast<uint16_t *>(reinterpret_cast<uint8_t *>(u.table) + table_bytes(p.kv.batch));
        const long long head = static_cast<long long>(u.cap) * p.kv.head_dim, page = head * p.kv.kv_heads;
        u.v = u.k + page * p.kv.batch;
        if (const cudaError_t e = launch_kv4_read(u, num_sms, stream); e != cudaSuccess)
            return e;
        AttnParams q = p;
        q.kv.k = u.k;
        q.kv.v = u.v;
        q.kv.block_table = u.table;
        q.kv.page_stride = page;
        q.kv.slot_stride = p.kv.head_dim;
        q.kv.head_stride = head;
        q.kv.num_pages = p.kv.batch;
        q.kv.page_size = u.cap;
        q.kv.blocks = 1;
        q.by_page = fast_div(u.cap);
        attn_set_tma(q);
        const cudaError_t e = launch_attn_chunk(q, grid, stream);
        if (e != cudaSuccess || p.whole)
            return e;
        return launch_attn_join(q, grid, false, static_cast<int>(std::min(static_cast<long long>(p.tile_rows), q_rows)), stream);
    }
    const cudaError_t e = few ? launch_kv4_decode(p, grid, stream) : launch_kv4_chunk(p, grid, stream);
    if (e != cudaSuccess || p.whole)
        return e;
    return launch_attn_join(p, grid, few, static_cast<int>(std::min(static_cast<long long>(p.tile_rows), q_rows)), stream);
}

}  // namespace qmm
