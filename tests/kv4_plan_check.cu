// Prints what qmm_kv4_attn would launch for batches read from stdin, one per line:
//   "batch tokens q_heads kv_heads head_dim page_size blocks window sinks max_q max_kv q_map more"
// (more: with the scratch to convert the keys once; few is 2 where it is used)
// Output per line: "few grid warps cluster whole unsplit tile_rows row_tiles min_chunk window
// sinks part_end", part_end the bytes of scratch the launch may touch, and the bytes asked
// for.  The launches and everything that asks the device are replaced here; host code only: it
// runs without a GPU.  tests/test_kv4_plan.py checks the answers.
#include <cstdio>
#include <cstring>

#include "../bit_weight_quantized_gb300/csrc/kv4_attn.cu"

namespace qmm {

static int q_map;

static void print_launch(const Kv4AttnParams &p, int grid, int few)
{
    const long long parts = p.whole ? 0 : 2LL * grid * (few ? kDecodeRows : kChunkRows) * p.kv.head_dim * 4;
    const long long end = p.whole ? 0 : static_cast<long long>(reinterpret_cast<uintptr_t>(p.part_o)) + parts;
    std::printf("%d %d %d %d %d %d %d %d %d %d %d %lld\n", few, grid, p.warps, p.cluster, p.whole, p.unsplit, p.tile_rows,
                p.row_tiles, p.min_chunk, p.window, p.sinks, end);
}

cudaError_t launch_kv4_decode(const Kv4AttnParams &p, int grid, cudaStream_t)
{
    print_launch(p, grid, 1);
    return cudaErrorUnknown;   // no joining kernel
}

cudaError_t launch_kv4_chunk(const Kv4AttnParams &p, int grid, cudaStream_t)
{
    print_launch(p, grid, 0);
    return cudaErrorUnknown;
}

// converted keys, read in 16 bits: the scratch ends behind them
static long long converted_end;
cudaError_t launch_kv4_read(Kv4ReadParams &p, int, cudaStream_t)
{
    converted_end = static_cast<long long>(reinterpret_cast<uintptr_t>(p.v)) +
                    2LL * p.kv.batch * p.kv.kv_heads * p.cap * p.kv.head_dim;
    return cudaSuccess;
}

cudaError_t launch_attn_chunk(const AttnParams &p, int grid, cudaStream_t)
{
    const long long parts = p.whole ? 0 : 2LL * grid * kChunkRows * p.kv.head_dim * 4 + reinterpret_cast<long long>(p.part_o);
    const bool apart = parts <= reinterpret_cast<long long>(p.kv.block_table);
    std::printf("2 %d %d %d %d %d %d %d %d %d %d %lld\n", grid, p.warps, p.cluster, p.whole, p.unsplit, p.tile_rows, p.row_tiles,
                p.min_chunk, p.window, p.sinks, apart ? converted_end : -1LL);
    return cudaErrorUnknown;
}

void attn_set_tma(AttnParams &p) { p.box = 0; }
cudaError_t launch_attn_join(const AttnParams &, int, bool, int, cudaStream_t) { return cudaErrorUnknown; }

// clusters that run at once, as 152 SMs would have them in parts of 16
int kv4_decode_clusters(int, bool, int rows, int cluster) { return (rows == 8 ? 288 : 144) / cluster; }
bool attn_set_q_tma(AttnParams &p) { return q_map != 0 && p.group <= 128; }

}  // namespace qmm

int main()
{
    using namespace qmm;
    int batch, tokens, hq, hk, D, page, blocks, window, sinks, max_q, max_kv, more;
    while (std::scanf("%d %d %d %d %d %d %d %d %d %d %d %d %d", &batch, &tokens, &hq, &hk, &D, &page, &blocks, &window, &sinks,
                      &max_q, &max_kv, &q_map, &more) == 13) {
        Kv4AttnParams p;
        std::memset(&p, 0, sizeof(p));
        p.kv.batch = batch;
        p.kv.tokens = tokens;
        p.kv.kv_heads = hk;
        p.kv.head_dim = D;
        p.kv.page_size = page;
        p.kv.blocks = blocks;
        p.q_heads = hq;
        p.group = hq / hk;
        p.causal = 1;
        p.window = window;
        p.sinks = sinks;
        const size_t extra = more ? kv4_attn_unpack_bytes(batch, tokens, p.group, hk, D, max_q, max_kv, sinks) : 0;
        kv4_attn_dispatch(p, max_q, max_kv, nullptr, extra, 152, nullptr);
        std::printf("%zu\n", kv4_attn_workspace_bytes(hq, hk, D, max_q, 152) + extra);
    }
    return 0;
}
