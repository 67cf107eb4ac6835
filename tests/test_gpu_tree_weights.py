"""Tree attention where weights, value scales or scores are not alike: a token that holds nearly all of the weight,
value scales far apart, places that some rows see and others do not, a negative scale.

The bound of an output row is the one of test_gpu_paged: every weight carries its own relative error (2^-11 of it, 2^-21
where it is kept in two parts, and what the rounded queries move its score by), so the row is off by that share of
sum p |v|, however the weights and the value scales are spread."""
import math

import numpy as np
import pytest
import torch

import paged_ref as ref
import rotational_w4a4_quantization_gb300 as rq
from test_gpu_paged import DEV, DTYPES, SEED, _built, _status, dev_cache, gen, paged, randn  # noqa: F401

pytestmark = pytest.mark.gpu
HALVES = [torch.bfloat16, torch.float16]
# query heads to a KV head, nodes: blocks of 8 and 16 rows, of 128, and (bf16) of 256
ROWS = [(1, 5), (4, 4), (4, 12), (4, 40)]


def pack(codes):
    """int codes [..., D] -> packed nibbles [..., D/2]"""
    c = codes.to(torch.int64) & 15
    return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8)


def check(q, cache, table, contexts, counts, scale, mask=None, rows=None, seen=None):
    """Against 64 bits, on the rows that `rows` names.  seen: the cache as far as it decides those rows (without what
    they do not see or what has no weight: 0 times infinity is no number, and a score that does not count may be off).
    Returns the output."""
    D = q.shape[-1]
    seen = dev_cache(cache if seen is None else seen)
    offsets = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)
    ctx = torch.tensor(contexts, dtype=torch.int32)
    cache, table, q = dev_cache(cache), table.to(DEV), q.to(DEV)
    got = rq.attn_tree(q, cache, table, ctx.to(DEV), offsets.to(DEV), SEED, 1, max_nodes=max(counts),
                       tree_mask=None if mask is None else mask.to(DEV), softmax_scale=scale)
    want, spread, delta = ref.attention_blocks(q, seen, table, contexts, offsets, SEED, 1,
                                               D ** -0.5 if scale is None else scale, mask)
    part = 2.0**-22 if q.dtype == torch.float32 else 2.0**-12
    folded = 2 if q.dtype == torch.bfloat16 and max(counts) * q.shape[1] // cache["kq"].shape[1] > 32 else 1
    eps = 8e-6 + folded * (2 * part + 2 * (4 / 3) * part * delta)
    bound = eps * spread.norm(dim=-1) + ref.UNIT[q.dtype] * want.norm(dim=-1) + (2.0**-25 * D**0.5 if q.dtype == torch.float16 else 0)
    err = (got.double() - want).norm(dim=-1)
    if rows is not None:
        err, bound = err[rows], bound[rows]
    assert (err <= bound).all(), (float((err / bound.clamp_min(1e-300)).max()), float((err / want.norm(dim=-1).max()).max()))
    return got


def aligned(N, H, G, n, D, dtype, seed, page=64):
    """One sequence of N tokens and n nodes whose queries lie along one direction: (q, cache, table, codes of the
    direction, length of a score of one code step).  The keys' codes are random, their scales 0 (to be set)."""
    g = gen(seed)
    along = torch.randint(3, 8, (D,), generator=g) * (2 * torch.randint(0, 2, (D,), generator=g) - 1)
    R = ref.rotation(D, SEED, 1)
    length = 0.9 + 0.2 * torch.rand(n, H * G, 1, generator=g, dtype=torch.float64)
    q = (length * (along.double() @ R.T) * (1.0 / D ** 0.5)).to(dtype)
    cache, table = paged([N + n], H, page, D, seed + 1)
    pages = cache["kq"].shape[0]
    cache["kq"] = pack(torch.randint(-7, 8, (pages, H, page, D), generator=g))
    step = float((along.double() ** 2).sum()) / D ** 0.5 * D ** -0.5        # the aligned key's score with scale 1
    return q, cache, table, along, step


def put(cache, table, page, at, name, codes=None, scale=None):
    pg, row = table[0].long()[at // page], at % page
    if codes is not None:
        cache[name + "q"][pg, :, row] = pack(codes)
    if scale is not None:
        cache[name + "s"][pg, :, row] = scale


@pytest.mark.parametrize("G,n", ROWS)
@pytest.mark.parametrize("dtype,bits,value", [(d, *w) for d in DTYPES for w in ((10, 1e-3), (14, 1e-3), (17, 0.0), (24, 0.0), (26, 0.0))]
                         + [(d, 45, 0.0) for d in DTYPES])
@pytest.mark.parametrize("first", [True, False])
def test_one_token_holds_the_weight(G, n, dtype, bits, value, first):
    """A token whose value row is small or nothing, `bits` bits of weight above each of 32k others, whose values have a
    common part."""
    N, H, D, page = 32768, 1, 128, 64
    q, cache, table, along, step = aligned(N, H, G, n, D, dtype, 400 + bits)
    g = gen(401)
    cache["ks"] = (0.3 + 0.2 * torch.rand(cache["ks"].shape, generator=g)) * (5.0 / step)     # scores within a few of 0
    pages = cache["kq"].shape[0]
    cache["vq"] = pack(3 + torch.randint(-3, 4, (pages, H, page, D), generator=g))
    cache["vs"] = 0.2 + 0.2 * torch.rand(cache["vs"].shape, generator=g)
    at = torch.tensor([0 if first else N - 200])
    put(cache, table, page, at, "k", along, bits * math.log(2) / step)
    put(cache, table, page, at, "v", None, value)
    check(q, cache, table, [N], [n], None)


@pytest.mark.parametrize("G,n", ROWS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("every", [16, 1000])
def test_large_values_of_no_weight(G, n, dtype, D, every):
    """Tokens whose value scale is 2^20 times the others' and whose weight is 2^-40 of theirs: the others' values
    decide the output."""
    N, H, page = 16384, 2, 64
    q, cache, table, along, step = aligned(N, H, G, n, D, dtype, 410)
    g = gen(411)
    cache["ks"] = (0.3 + 0.2 * torch.rand(cache["ks"].shape, generator=g)) * (5.0 / step)
    cache["vs"] = 2e-2 * (0.5 + torch.rand(cache["vs"].shape, generator=g))
    at = torch.arange(3, N, every)
    put(cache, table, page, at, "k", -along, 40 * math.log(2) / step)
    put(cache, table, page, at, "v", None, 2e-2 * 2.0**20)
    check(q, cache, table, [N], [n], None)


@pytest.mark.parametrize("G,n", ROWS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bits", [6, 13, 20, 30])
def test_value_scales_apart(G, n, dtype, bits):
    """Value scales spread over `bits` bits in every tile, the small ones where the weight is."""
    N, H, D, page = 16384, 2, 128, 64
    q, cache, table, along, step = aligned(N, H, G, n, D, dtype, 420)
    g = gen(421)
    down = torch.randint(0, bits + 1, (N,), generator=g).float()
    at = torch.arange(N)
    put(cache, table, page, at, "k", (along[None, :] * torch.where(down > 0, 1, -1)[:, None])[:, None, :].expand(-1, H, -1),
        ((1.5 * down - 1).abs() * math.log(2) / step)[:, None])
    put(cache, table, page, at, "v", None, (0.3 * torch.exp2(-down))[:, None])
    check(q, cache, table, [N], [n], None)


@pytest.mark.parametrize("G,n", [(4, 12), (4, 40)])
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("bits", [13, 20, 27])
def test_key_scales_apart(G, n, dtype, bits):
    """One key per tile with a scale 2^bits above the others', far below them in score: the others' scores decide."""
    N, H, D, page = 16384, 2, 128, 64
    q, cache, table, along, step = aligned(N, H, G, n, D, dtype, 430)
    g = gen(431)
    small = 20.0 / step
    cache["ks"] = (0.3 + 0.2 * torch.rand(cache["ks"].shape, generator=g)) * small
    at = torch.arange(5, N, 100)
    put(cache, table, page, at, "k", -along, small * 2.0**bits)
    seen = {name: t.clone() for name, t in cache.items()}
    put(seen, table, page, at, "k", -along, 40.0 / step)              # e^-40 of the others' weight as well
    check(q, cache, table, [N], [n], None, seen=seen)


@pytest.mark.parametrize("G,n,dtype", [(4, 12, torch.bfloat16), (4, 40, torch.bfloat16), (4, 12, torch.float16), (1, 5, torch.bfloat16)])
@pytest.mark.parametrize("zero", [(0, 128), (128, 256), (256, 640)])
def test_tiles_of_zero_values(G, n, dtype, zero):
    """Whole tiles of zero value rows before and between tiles of small values."""
    B, H, D, page = 16, 2, 128, 64
    contexts, counts = [700 + 5 * b for b in range(B)], [n] * B
    cache, table = paged([c + n for c in contexts], H, page, D, 440)
    cache["vs"] *= 1e-9 if dtype == torch.bfloat16 else 2e-3
    at = torch.arange(*zero)
    for b in range(B):
        cache["vs"][table[b].long()[at // page], :, at % page] = 0.0
    check(randn(B * n, H * G, D, seed=441, dtype=dtype), cache, table, contexts, counts, None)


@pytest.mark.parametrize("G,n", [(1, 7), (1, 13), (4, 3), (4, 12), (4, 40)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [float("inf"), 3e38, 2.0**20, float("nan")])
def test_a_place_that_only_some_rows_see(G, n, dtype, scale):
    """Nodes 0 and 1 hold a value scale that is infinite, huge or no number; rows that see neither are as if it were not there."""
    B, H, D, page = 80, 1, 64, 32
    g = gen(450)
    contexts, counts = torch.randint(40, 150, (B,), generator=g).tolist(), [n] * B
    cache, table = paged([c + n for c in contexts], H, page, D, 451)
    mask = torch.zeros(B * n, n, dtype=torch.bool)
    for i in range(B * n):
        mask[i] = torch.rand(n, generator=g) < 0.4
        mask[i, i % n] = True
        if i % n not in (0, 1):
            mask[i, :2] = torch.rand(1, generator=g) < 0.3
    sees = mask[:, :2].any(1)
    seen = {name: t.clone() for name, t in cache.items()}
    for b, c in enumerate(contexts):
        for j in range(2):
            pg, row = int(table[b, (c + j) // page]), (c + j) % page
            cache["vs"][pg, :, row] = scale
    rows = ~sees.to(DEV)
    got = check(randn(B * n, H * G, D, seed=452, dtype=dtype), cache, table, contexts, counts, None, mask, rows, seen)
    assert torch.isfinite(got[rows]).all()


@pytest.mark.parametrize("G,n", [(1, 5), (4, 4), (4, 12), (4, 40)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [-0.3, -1e-3])
def test_negative_scale(G, n, dtype, scale):
    """The softmax of negative multiples of the scores; contexts that end inside a tile, a mask."""
    B, H, D, page = 80, 1, 128, 32
    g = gen(460)
    contexts, counts = torch.randint(1, 150, (B,), generator=g).tolist(), [n] * B
    cache, table = paged([c + n for c in contexts], H, page, D, 461)
    check(randn(B * n, H * G, D, seed=462, dtype=dtype), cache, table, contexts, counts, scale, ref.tree_mask(counts, g))
