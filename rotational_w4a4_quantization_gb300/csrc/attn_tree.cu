// attn_tree.cu -- tree attention over the paged cache: which kernel a call takes, and its
// workspace.
#include "attn_tree_mma.cuh"

namespace rq {

int64_t attn_tree_workspace(int64_t head_dim) {
    const int sms = device_sm_count();
    int64_t most = attn_tree_tc_workspace(head_dim);
    for (int rows = 8; rows <= 16; rows *= 2) {
        const int ctas = blocks_per_sm(rows, head_dim) * sms;
        const int64_t bytes = tree_join_at(ctas, rows, (int)head_dim) * (int64_t)sizeof(float) + ctas * (int64_t)sizeof(TreeJoin);
        if (bytes > most) most = bytes;
    }
    return most;
}

cudaError_t launch_attn_tree(const TreeCall &c, cudaStream_t stream) {
    if (attn_tree_tc_supported(c)) return launch_attn_tree_tc(c, stream);
    TreeParams p;
    if (!tree_params(c, p)) return cudaErrorUnknown;
    return launch_tree_mma(c, p, stream);
}

}  // namespace rq
