// attn_tree_tc.cu -- tree attention on the 5th-generation tensor cores: which calls it takes,
// and its workspace.
#include "attn_tree_tc.cuh"

namespace rq {

// Blocks of 128 rows pay a long start and end per unit, blocks of 16 rows more per token and
// row.  Measured (8 KV heads x 128, cold caches), here and there: 16 sequences of 4k, bf16,
// 32 rows 70 and 58 us, 48 rows 72 and 81, 64 rows 73 and 101; 64 of 300, 32 rows 64 and 59,
// 48 rows 68 and 79; fp16, 4 of 32k, 32 rows 113 and 102, 48 rows 114 and 142.  Where there
// are fewer tiles than SMs either does (2 of 512, 64 rows: 18 and 20).  The rows are those
// that there are on average, the tiles as many as the table can name.
bool attn_tree_tc_supported(const TreeCall &c) {
    const int64_t rows = tree_rows(c), tiles = tree_tiles(c, 128, kTcTT);
    return c.in_type != IN_F32 && (c.head_dim == 64 || c.head_dim == 128) && rows > 32 && tiles > device_sm_count();
}

int64_t attn_tree_tc_workspace(int64_t head_dim) {
    if (head_dim != 64 && head_dim != 128) return 0;
    const int sms = device_sm_count();
    return tree_join_at(sms, 256, (int)head_dim) * (int64_t)sizeof(float) + sms * (int64_t)sizeof(TreeJoin);
}

cudaError_t launch_attn_tree_tc(const TreeCall &c, cudaStream_t stream) {
    TreeParams p;
    if (!tree_params(c, p)) return cudaErrorUnknown;
    return launch_tree_tc(c, p, stream);
}

}  // namespace rq
