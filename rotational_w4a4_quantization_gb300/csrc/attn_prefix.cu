// attn_prefix.cu -- attention of sequences that share a prefix, over the paged rotated INT4
// cache (sm_103a).
//
//   out = softmax([e_prefix, e_own]) [v^_prefix; v^_own] R^T
// with the scores of attn_tree_mma.cuh.  The softmax over both is that of either with its
// reference z and sum l, joined:  z = max(z1, z2), l = l1 2^(z1 - z) + l2 2^(z2 - z), and O
// alike.  So the prefix is read once for a block of all its group's rows: a first pass takes the groups
// for sequences, with the rows of all their sequences as nodes that see every token, and
// leaves O, z and l of each row in fp32; the second goes over each sequence's own tokens and
// begins each row from there.  Both are the kernels of tree attention, which choose their
// blocks by the rows of the pass.  The second needs the first's rows only where it finishes its
// own, so it begins beside the first's end, with scratch of its own.  Blocks of few rows join
// the partials that the first pass has left of each of their rows by themselves: its units
// note for each row where those are.  Blocks of many rows find them joined in the state.
//
// Measured, bf16, heads of 128, one token a sequence, in a graph on the same inputs (and after a
// flush of L2, which takes the kernels' code with it): 64 sequences with one prompt of 8k and up to
// 512 own tokens, 32 heads on 8, 48 us (61); 256 sequences with two prompts of up to 32k and up to
// 2k own tokens, 64 heads on 8, 372 us (375); 4 sequences with 1000 + 37 tokens, fp16, 16 us (26).
// Those are with tables of the longest sequence's width; with tables for 64k tokens the first take
// 53 us, on blocks of 256 rows, the last 25, with a join behind the second pass.  The first pass is
// bound by the softmax of its blocks of many rows, the second by its units' starts and ends, some 8 us
// each, then by the codes.  Both wait for registers now and then: with 168 or 128 of them the
// instances for heads of 128 spill 36 to 72 bytes a thread (fp32 68 to 136), those on tensor
// cores, of 96, 20 to 52; tree attention's own 12 to 68, fp32 32 to 96, and 20 to 40.
#include "attn_tree_mma.cuh"

namespace rq {
namespace {

cudaError_t launch_tree_pass(TreePass &pass, cudaStream_t stream) {
    if (attn_tree_tc_supported(pass.call)) return launch_tree_pass_tc(pass, stream);
    TreePassParams p;
    if (!tree_params(pass, p)) return cudaErrorUnknown;
    const cudaError_t e = launch_tree_mma(pass.call, p, stream);
    pass.out_rows = p.out_rows;
    pass.out_ctas = p.ctas;
    return e;
}

}  // namespace

// Each pass's scratch (a multiple of 16 bytes), then the state, then the rows' places.
int64_t attn_prefix_workspace(int64_t rows, int64_t q_heads, int64_t head_dim) {
    return 2 * attn_tree_workspace(head_dim) + rows * q_heads * (int64_t)(sizeof(TreePlace) + (head_dim + 2) * sizeof(float));
}

cudaError_t launch_attn_prefix(const TreeCall &c, const PrefixCall &prefix, cudaStream_t stream) {
    char *const scratch = static_cast<char *>(c.workspace);
    const int64_t each = attn_tree_workspace(c.head_dim);
    float *const state = reinterpret_cast<float *>(scratch + 2 * each);
    void *const place = state + c.rows * c.q_heads * (c.head_dim + 2);
    TreePass first{c, prefix.groups, c.seqs, state}, second{c, nullptr, 0, state};
    first.call.table = prefix.table;
    first.call.width = prefix.width;
    first.call.contexts = prefix.lens;
    first.call.seqs = prefix.n_groups;
    first.call.max_nodes = c.rows;
    first.call.mask = nullptr;
    second.call.workspace = scratch + each;
    // blocks of few rows join the first pass's partials as they take their rows up
    if (!attn_tree_tc_supported(second.call)) first.place = second.place = place;
    cudaError_t e = launch_tree_pass(first, stream);
    if (e != cudaSuccess) return e;
    second.out_part = static_cast<const float *>(first.call.workspace);
    second.out_rows = first.out_rows;
    second.out_ctas = first.out_ctas;
    return launch_tree_pass(second, stream);
}

}  // namespace rq
