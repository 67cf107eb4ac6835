// attn_prefix_tc.cu -- a pass of shared-prefix attention (see attn_prefix.cu) on the
// 5th-generation tensor cores.
#include "attn_tree_tc.cuh"

namespace rq {

cudaError_t launch_tree_pass_tc(TreePass &pass, cudaStream_t stream) {
    TreePassParams p;
    if (!tree_params(pass, p)) return cudaErrorUnknown;
    const cudaError_t e = launch_tree_tc(pass.call, p, stream);
    pass.out_rows = p.out_rows;
    pass.out_ctas = p.ctas;
    return e;
}

}  // namespace rq
