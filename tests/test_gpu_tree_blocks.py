"""Tree attention by kind of row block: 8 and 16 rows (mma.sync), 128 and 256 rows (tcgen05, which takes 16-bit
queries of more than 32 rows per KV head where there are more tiles than SMs)."""
import numpy as np
import pytest
import torch

import paged_ref as ref
import rotational_w4a4_quantization_gb300 as rq
from test_gpu_paged import DEV, DTYPES, SEED, _built, _status, check_tree, dev_cache, gen, paged, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("G,n", [(1, 7), (2, 4), (8, 1), (3, 3), (16, 1), (17, 1), (1, 17)])
def test_rows_around_the_blocks(dtype, D, G, n):
    """7, 8, 9, 16 and 17 rows per KV head."""
    counts, contexts = [n, 1, max(1, n - 1)], [40, 513, 190]
    cache, table = paged([c + k for c, k in zip(contexts, counts)], 2, 16, D, 200 + n)
    q = randn(sum(counts), 2 * G, D, seed=201, dtype=dtype)
    check_tree(q, cache, table, contexts, counts, mask=ref.tree_mask(counts, gen(202)), max_nodes=n)


def check_large(q, cache, table, contexts, counts, mask, scale):
    """check_tree's bound, with k^ and v^ rounded to fp16 as well (once each, as q~ and the weights) for bf16."""
    D = q.shape[-1]
    ctx = torch.tensor(contexts, dtype=torch.int32)
    offsets = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)
    got = rq.attn_tree(q.to(DEV), dev_cache(cache), table.to(DEV), ctx.to(DEV), offsets.to(DEV), SEED, 1,
                       tree_mask=mask.to(DEV), softmax_scale=scale)
    want, spread, delta = ref.attention(q, cache, table, ctx, offsets, SEED, 1, D ** -0.5 if scale is None else scale, mask)
    g = got.cpu().double()
    assert torch.isfinite(g).all()
    times = 2 if q.dtype == torch.bfloat16 else 1
    eps = 8e-6 + times * 2.0**-11 * (1 + (4 / 3) * delta)
    bound = eps * spread.norm(dim=-1) + ref.UNIT[q.dtype] * want.norm(dim=-1) + (2.0**-25 * D**0.5 if q.dtype == torch.float16 else 0)
    err = (g - want).norm(dim=-1)
    assert (err <= bound).all(), float((err / bound.clamp_min(1e-300)).max())
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,D", [(12, 128), (40, 128), (12, 64), (40, 64)])
@pytest.mark.parametrize("kind", ["plain", "sharp", "flat", "tiny_values", "huge_values", "uneven_values", "uneven_keys",
                                  "large_queries", "poison"])
def test_large_blocks(dtype, n, D, kind):
    B, G, page = 80, 4, 32
    g = gen(210)
    contexts = torch.randint(131, 150, (B,), generator=g).tolist()
    counts = torch.randint(1, n + 1, (B,), generator=g).tolist()
    counts[0], counts[1], contexts[2], contexts[3] = n, n, 0, 1
    counts[4] = 0
    cache, table = paged([c + k for c, k in zip(contexts, counts)], 1, page, D, 211)
    mask = ref.tree_mask(counts, g)
    mask = torch.nn.functional.pad(mask, (0, n - mask.shape[1]))
    scale, qs = None, 1.0
    half = dtype == torch.float16
    if kind == "sharp":
        scale = 0.6
    if kind == "flat":
        scale = 0.0
    if kind == "tiny_values":
        cache["vs"] *= 1e-2 if half else 1e-9
    if kind == "huge_values":
        cache["vs"] *= 1e3 if half else 1e9
    if kind == "uneven_values":
        cache["vs"] *= torch.exp2(-20.0 * torch.rand(cache["vs"].shape, generator=g))
    if kind == "uneven_keys":
        cache["ks"] *= torch.exp2(-20.0 * torch.rand(cache["ks"].shape, generator=g))
    if kind == "large_queries":
        scale, qs = 1e-4, 3000.0
    starts = np.cumsum([0] + counts)
    if kind == "poison":
        mask[:, 0] = False                                      # node 0 is hidden from all, so are roots' rows
        mask[starts[2]:starts[3]] = False                       # nothing visible: context 0
        used = torch.zeros(cache["ks"].shape[0], page, dtype=torch.bool)
        for b, (c, k) in enumerate(zip(contexts, counts)):
            pg, row = ref.places(table, page, b, c + k)
            used[pg, row] = True
            if b == 2:
                used[pg, row] = False
            elif k:
                used[pg[c], row[c]] = False
        for name in ("ks", "vs"):
            bad = torch.tensor([float("nan"), float("inf"), float("-inf"), 3e38])
            t = cache[name].transpose(1, 2)
            t[~used] = bad[torch.arange(int((~used).sum())) % 4][:, None]
    q = randn(sum(counts), G, D, seed=212, dtype=dtype, scale=qs)
    got = check_large(q, cache, table, contexts, counts, mask, scale)
    if kind == "poison":
        assert (got[starts[2]:starts[3]] == 0).all()
