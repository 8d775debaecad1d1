// Prints what qmm_paged_attn would launch for batches read from stdin, one per line:
//   "batch tokens q_heads kv_heads head_dim page_size blocks window max_q max_kv q_map"
// (q_map: 1 where the queries take a tensor map).  Output per line: "few grid warps
// cluster whole unsplit tile_rows row_tiles min_chunk window part_end", part_end the bytes of
// scratch the launch may touch, and the bytes asked for.  With the argument "start" the lines
// are "position window" and the answers the first visible keys.  The attention kernels' launches and
// everything that asks the device are replaced here; host code only: it runs without
// a GPU.  tests/test_paged_plan.py checks the answers.
#include <cstdio>
#include <cstring>

#include "../bit_weight_quantized_gb300/csrc/attn.cu"

namespace qmm {

static int q_map;

static void print_launch(const AttnParams &p, int grid, int few)
{
    const long long parts = p.whole ? 0 : 2LL * grid * (few ? kDecodeRows : kChunkRows) * p.kv.head_dim * 4;
    const long long end = p.whole ? 0 : static_cast<long long>(reinterpret_cast<uintptr_t>(p.part_o)) + parts;
    std::printf("%d %d %d %d %d %d %d %d %d %d %lld\n", few, grid, p.warps, p.cluster, p.whole, p.unsplit, p.tile_rows,
                p.row_tiles, p.min_chunk, p.window, end);
}

cudaError_t launch_attn_decode(const AttnParams &p, int grid, cudaStream_t)
{
    print_launch(p, grid, 1);
    return cudaErrorUnknown;   // no joining kernel
}

cudaError_t launch_attn_chunk(const AttnParams &p, int grid, cudaStream_t)
{
    print_launch(p, grid, 0);
    return cudaErrorUnknown;
}

// clusters that run at once, as 152 SMs would have them in parts of 16
int attn_decode_clusters(int, bool, int warps, int cluster) { return (warps == 8 ? 144 : 288) / cluster; }
void attn_set_tma(AttnParams &p) { p.box = 0; }
bool attn_set_q_tma(AttnParams &p) { return q_map != 0 && p.group <= 128; }

}  // namespace qmm

int main(int argc, char **argv)
{
    using namespace qmm;
    if (argc > 1 && !std::strcmp(argv[1], "start")) {
        int pos, w;
        while (std::scanf("%d %d", &pos, &w) == 2)
            std::printf("%d\n", window_start(pos, w));
        return 0;
    }
    int batch, tokens, hq, hk, D, page, blocks, window, max_q, max_kv;
    while (std::scanf("%d %d %d %d %d %d %d %d %d %d %d", &batch, &tokens, &hq, &hk, &D, &page, &blocks, &window, &max_q,
                      &max_kv, &q_map) == 11) {
        AttnParams p;
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
        attn_dispatch(p, max_q, max_kv, nullptr, 152, nullptr);
        std::printf("%zu\n", attn_workspace_bytes(hq, hk, D, max_q, 152));
    }
    return 0;
}
