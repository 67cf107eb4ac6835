"""Tree attention in a captured graph: a replay gives the call's bits, also to what follows it."""
import numpy as np
import pytest
import torch

import paged_ref as ref
import rotational_w4a4_quantization_gb300 as rq
from test_gpu_paged import DEV, SEED, _built, _status, check_tree, dev_cache, gen, paged, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,H,G,n,context,D", [
    (1, 2, 4, 1, 60, 128),       # every unit in one block: the join has nothing to do
    (200, 2, 4, 1, 90, 64),
    (200, 2, 4, 12, 90, 128),    # the same, blocks of 128 rows
    (2, 4, 4, 5, 3000, 128),     # units over many blocks
    (16, 8, 4, 40, 700, 64),
])
def test_replay_gives_the_calls_bits(B, H, G, n, context, D):
    g = gen(300 + B)
    contexts = torch.randint(context // 2, context + 1, (B,), generator=g).tolist()
    cache, table = paged([c + n for c in contexts], H, 32, D, 301)
    counts = [n] * B
    mask = ref.tree_mask(counts, g)
    qs = [randn(B * n, H * G, D, seed=302 + i, dtype=torch.bfloat16) for i in range(2)]
    wants = [check_tree(q, cache, table, contexts, counts, mask=mask) if B < 50 else None for q in qs]
    dc, tb, m = dev_cache(cache), table.to(DEV), mask.to(DEV)
    ctx = torch.tensor(contexts, dtype=torch.int32, device=DEV)
    off = torch.arange(0, B * n + 1, n, dtype=torch.int32, device=DEV)
    call = lambda q, **kw: rq.attn_tree(q, dc, tb, ctx, off, SEED, 1, tree_mask=m, **kw)
    wants = [call(q.to(DEV)).clone() if w is None else w for q, w in zip(qs, wants)]
    assert all(torch.isfinite(w).all() for w in wants)
    q, out = qs[0].to(DEV), torch.empty_like(wants[0])
    ws = torch.empty(rq.attn_tree_workspace(D), dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call(q, out=out, workspace=ws)                        # what is loaded on the first call
        copy = torch.empty_like(out)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call(q, out=out, workspace=ws)
        copy.copy_(out)                                       # ordered behind the join alone
    for i in (0, 1, 0, 1):
        q.copy_(qs[i])
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(copy, wants[i]) and torch.equal(out, wants[i])
