"""Tree attention with bounds that say little: max_nodes left out or large, masks wider than the trees, block tables
as wide as the longest context that a server allows.  They choose neither the results nor the schedule."""
import numpy as np
import pytest
import torch

import paged_ref as ref
import rotational_w4a4_quantization_gb300 as rq
from test_gpu_paged import DEV, DTYPES, SEED, _built, _status, dev_cache, gen, paged, randn  # noqa: F401

pytestmark = pytest.mark.gpu


def batch(B, H, G, n, context, D, dtype, page=64, seed=500):
    g = gen(seed)
    contexts = torch.randint(context // 2, context + 1, (B,), generator=g).tolist()
    cache, table = paged([c + n for c in contexts], H, page, D, seed + 1)
    q = randn(B * n, H * G, D, seed=seed + 2, dtype=dtype).to(DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    return q, dev_cache(cache), table.to(DEV), i32(contexts), i32([b * n for b in range(B + 1)])


def micros(f):
    f()
    times = []
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(5):
            f()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 200.0)
    return sorted(times)[2]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,n,G", [(300, 1, 8), (40, 3, 4), (64, 12, 4)])
def test_without_max_nodes(dtype, B, n, G):
    """A batch without a mask that leaves max_nodes out, against 64 bits; with sequences of no nodes."""
    D = 64
    q, cache, table, ctx, off = batch(B, 2, G, n, 150, D, dtype)
    off[5:] -= n                                             # the fifth has none, and every later one's rows move up
    rows = int(off[-1])
    q = q[:rows]
    got = rq.attn_tree(q, cache, table, ctx, off, SEED)
    want, spread, delta = ref.attention_blocks(q, cache, table.cpu(), ctx.tolist(), off, SEED, 1, D ** -0.5)
    part = 2.0**-22 if dtype == torch.float32 else 2.0**-12
    eps = 8e-6 + (2 if dtype == torch.bfloat16 else 1) * (2 * part + 2 * (4 / 3) * part * delta)
    bound = eps * spread.norm(dim=-1) + ref.UNIT[dtype] * want.norm(dim=-1) + (2.0**-25 * D**0.5 if dtype == torch.float16 else 0)
    assert ((got.double() - want).norm(dim=-1) <= bound).all()


def test_a_decode_batch_without_max_nodes_is_as_fast():
    """2048 sequences, one node each."""
    q, cache, table, ctx, off = batch(2048, 2, 8, 1, 200, 128, torch.bfloat16)
    exact = micros(lambda: rq.attn_tree(q, cache, table, ctx, off, SEED, max_nodes=1))
    left_out = micros(lambda: rq.attn_tree(q, cache, table, ctx, off, SEED))
    assert left_out < 1.5 * exact, (left_out, exact)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,H,G,n,context,D", [(64, 8, 8, 1, 1100, 128), (24, 8, 4, 3, 1900, 64), (24, 8, 4, 12, 1500, 128)])
def test_wide_bounds_keep_the_schedule(dtype, B, H, G, n, context, D):
    """A table 16 times as wide as the contexts need, max_nodes and mask far above the trees: the same bits."""
    q, cache, table, ctx, off = batch(B, H, G, n, context, D, dtype)
    mask = ref.tree_mask([n] * B, gen(510)).to(DEV)
    want = rq.attn_tree(q, cache, table, ctx, off, SEED, tree_mask=mask, max_nodes=n)
    wide = torch.full((B, 16 * table.shape[1]), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    assert torch.equal(want, rq.attn_tree(q, cache, wide, ctx, off, SEED, tree_mask=mask, max_nodes=n))
    large = torch.zeros(B * n, 200, dtype=torch.bool, device=DEV)
    large[:, :n] = mask
    assert torch.equal(want, rq.attn_tree(q, cache, table, ctx, off, SEED, tree_mask=large))
    assert torch.equal(want, rq.attn_tree(q, cache, wide, ctx, off, SEED, tree_mask=large))
