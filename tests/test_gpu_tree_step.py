"""The verification step that runs rope, kv_append, attn_tree and kv_read together."""
import pytest
import torch

import rotational_w4a4_quantization_gb300 as rq
from rotational_w4a4_quantization_gb300.tree_step import SEED, TreeStep

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs,context,nodes,heads,kv_heads,dim,page", [
    (1, 1, 1, 4, 4, 32, 16),
    (3, 130, 9, 8, 2, 128, 32),
    (24, 900, 40, 8, 4, 64, 64),       # rows enough for the larger blocks
])
def test_step_matches_64_bits(seqs, context, nodes, heads, kv_heads, dim, page):
    step = TreeStep(seqs, context, nodes, heads, kv_heads, dim, page)
    # bf16 rounds each element by up to 2^-8 of itself, weights and folded operands by 2^-11 or less
    assert step.error(*step.attend()) < 6e-3


def test_accepted_path_is_what_a_plain_write_leaves():
    """A path's tokens written again read back as if they had been the sequence from the start."""
    step = TreeStep(2, 50, 12, 4, 2, 64, 16)
    step.attend()
    path = torch.stack([step.mask[12 * b + 11].cpu().nonzero().flatten()[:2]
                        for b in range(2)]).to("cuda")
    step.accept(path)
    n = path.shape[1]
    offsets = torch.arange(3, dtype=torch.int32, device="cuda") * n
    starts = torch.full((2,), 50, dtype=torch.int32, device="cuda")
    k, v = rq.kv_read(step.cache, step.table, starts, offsets, 2 * n, SEED, dtype=torch.float32)
    cache = rq.kv_cache(1, 2, 64, 16)
    rows = (path + 12 * torch.arange(2, device="cuda")[:, None]).flatten()
    positions = (50 + torch.arange(n, device="cuda")).repeat(2)
    rq.kv_append(step.k[rows], step.v[rows], cache, torch.arange(2 * n, device="cuda"), SEED, positions=positions,
                 turns=step.turns)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    k1, v1 = rq.kv_read(cache, table, None, torch.tensor([0, 2 * n], dtype=torch.int32, device="cuda"), 2 * n, SEED,
                        dtype=torch.float32)
    assert torch.equal(k, k1) and torch.equal(v, v1)
