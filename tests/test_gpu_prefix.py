"""Shared-prefix attention against 64 bits over tables that name each sequence's prefix and own tokens, with the
tolerances of tree attention (test_gpu_paged; keys and values of bf16 queries in large blocks are rounded as well).  The two
passes are joined in fp32: a few roundings of 2^-24, within the 8e-6 that is there for fp32's part."""
import numpy as np
import pytest
import torch

import paged_ref
import prefix_ref as ref
import rotational_w4a4_quantization_gb300 as rq
from rotational_w4a4_quantization_gb300.prefix_step import PrefixStep
from test_gpu_paged import DEV, DTYPES, SEED, _built, _status, dev_cache, filled_cache, gen, randn  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32)


def tables(lengths, order, page):
    need = [-(-n // page) for n in lengths]
    t = torch.full((len(lengths), max(1, max(need, default=0))), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        t[b, :n] = torch.tensor(order[:n], dtype=torch.int32)
        order = order[n:]
    return t, order


def batch(sizes, prefixes, own, counts, H, page, D, seed):
    """Cache and tables of groups of `sizes` sequences with `prefixes`; own and counts by sequence."""
    lengths = [c + n for c, n in zip(own, counts)]
    pages = sum(-(-n // page) for n in lengths + list(prefixes)) + 2
    order = torch.randperm(pages, generator=gen(seed)).tolist()
    ptable, order = tables(prefixes, order, page)
    table, _ = tables(lengths, order, page)
    return filled_cache(pages, H, page, D, seed + 1), table, ptable, i32([0] + list(np.cumsum(sizes)))


def run(q, cache, table, ptable, groups, prefixes, own, counts, flags=1, mask=None, scale=None, max_nodes=None, **kw):
    d = lambda x: None if x is None else x.to(DEV)
    return rq.attn_prefix(d(q), dev_cache(cache), d(table), d(i32(own)), d(i32([0] + list(np.cumsum(counts)))), d(ptable),
                          d(i32(prefixes)), d(groups), SEED, flags, tree_mask=d(mask), softmax_scale=scale,
                          max_nodes=max_nodes or (None if mask is not None else max(counts)), **kw)


def check(q, cache, table, ptable, groups, prefixes, own, counts, flags=1, mask=None, scale=None, blocks=False, pad=0, **kw):
    D = q.shape[-1]
    if pad:                                                         # rows of no sequence: left as they were
        more = torch.cat([q, torch.full((pad, *q.shape[1:]), float("nan"), dtype=q.dtype)])
        out = torch.full(more.shape, 7.0, dtype=q.dtype, device=DEV)
        wide = None if mask is None else torch.cat([mask, torch.ones(pad, mask.shape[1], dtype=torch.bool)])
        got = run(more, cache, table, ptable, groups, prefixes, own, counts, flags, wide, scale, out=out, **kw)
        assert (got[-pad:] == 7.0).all()
        got = got[:-pad]
    else:
        got = run(q, cache, table, ptable, groups, prefixes, own, counts, flags, mask, scale, **kw)
    assert got.dtype == q.dtype and got.shape == q.shape
    flat, joint, ctx = ref.joined(cache, table, own, counts, ptable, prefixes, groups)
    offsets = i32([0] + list(np.cumsum(counts)))
    sc = D ** -0.5 if scale is None else scale
    if blocks:
        want, spread, delta = (x.cpu() for x in paged_ref.attention_blocks(q.to(DEV), dev_cache(flat), joint.to(DEV), ctx.tolist(),
                                                                           offsets, SEED, flags, sc, mask))
    else:
        want, spread, delta = paged_ref.attention(q, flat, joint, ctx, offsets, SEED, flags, sc, mask, rotated=bool(flags & 2))
    g = got.cpu().double()
    assert torch.isfinite(g).all()
    part = 2.0**-22 if q.dtype == torch.float32 else 2.0**-12
    rows = max(sum(counts[groups[i]:groups[i + 1]]) for i in range(len(prefixes))) * q.shape[1] // cache["kq"].shape[1]
    folded = 2 if q.dtype == torch.bfloat16 and rows > 32 else 1
    eps = 8e-6 + folded * (2 * part + 2 * (4 / 3) * part * delta)
    err = (g - want).norm(dim=-1)
    bound = eps * spread.norm(dim=-1) + paged_ref.UNIT[q.dtype] * want.norm(dim=-1) + (2.0**-25 * D**0.5 if q.dtype == torch.float16 else 0)
    assert (err <= bound).all(), float((err / bound.clamp_min(1e-300)).max())
    return got


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,page", [(32, 16), (64, 32), (128, 64), (256, 128)])
@pytest.mark.parametrize("H,G,n", [(2, 1, 1), (1, 4, 1), (2, 4, 3), (1, 8, 6)])
def test_shapes(dtype, D, page, H, G, n):
    sizes, prefixes = [3, 1, 2], [300, 64, 129]
    own, counts = [40, 0, 200, 5, 129, 31], [n, 1, n, max(1, n - 1), n, 1]
    cache, table, ptable, groups = batch(sizes, prefixes, own, counts, H, page, D, 400 + n)
    q = randn(sum(counts), H * G, D, seed=401, dtype=dtype)
    mask = paged_ref.tree_mask(counts, gen(402)) if n > 1 else None
    check(q, cache, table, ptable, groups, prefixes, own, counts, mask=mask)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 127, 128, 129, 2000])
@pytest.mark.parametrize("own", [0, 1, 130])
def test_lengths(dtype, prefix, own):
    """Prefixes that end inside a page and inside a tile, from none; a first own token without others."""
    H, G, D = 2, 4, 128
    cache, table, ptable, groups = batch([4], [prefix], [own, 0, own, 3], [1] * 4, H, 16, D, 410 + prefix)
    check(randn(4, H * G, D, seed=411, dtype=dtype), cache, table, ptable, groups, [prefix], [own, 0, own, 3], [1] * 4)


@pytest.mark.parametrize("flags", [0, 1, 2, 3])
@pytest.mark.parametrize("n,seqs", [(1, 3), (2, 24)])
def test_bases(flags, n, seqs):
    own, counts = [(13 * b) % 70 for b in range(seqs)], [n] * seqs
    cache, table, ptable, groups = batch([seqs], [150], own, counts, 2, 32, 64, 420)
    check(randn(n * seqs, 8, 64, seed=421, dtype=torch.float16), cache, table, ptable, groups, [150], own, counts, flags)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("seqs,G,prefix", [(40, 4, 3000), (70, 4, 2500), (9, 2, 6000), (150, 1, 300)])
def test_many_sequences_and_tiles(dtype, D, seqs, G, prefix):
    """Groups whose rows fill blocks of 16, 128 and 256, prefixes over many blocks; the second group has none, some
    sequences are in no group."""
    H, g = 8, gen(430)
    sizes, prefixes = [seqs - 5, 2, 1], [prefix, 0, 77]
    own = torch.randint(0, 200, (seqs,), generator=g).tolist()
    cache, table, ptable, groups = batch(sizes, prefixes, own, [1] * seqs, H, 64, D, 431)
    groups = groups + 1                                             # the first sequence and the last belong to none
    q = randn(seqs, H * G, D, seed=432, dtype=dtype)
    check(q, cache, table, ptable, groups, prefixes, own, [1] * seqs, blocks=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("seqs,n", [(2, 3), (30, 9)])
def test_trees_padding_and_empty_rows(dtype, seqs, n):
    """Trees of uneven size, sequences without nodes, rows of no sequence left as they were, rows whose mask leaves
    them the prefix alone."""
    g = gen(440)
    counts = torch.randint(1, n + 1, (seqs,), generator=g).tolist()
    counts[0], counts[1] = n, 0
    own = torch.randint(0, 90, (seqs,), generator=g).tolist()
    own[0] = 0
    cache, table, ptable, groups = batch([seqs], [333], own, counts, 2, 16, 64, 441)
    mask = paged_ref.tree_mask(counts, g, n)
    mask[:n] = False                                                # the first tree sees the prefix alone
    q = randn(sum(counts), 8, 64, seed=442, dtype=dtype)
    # the padded call splits its work by other rows, so that it has the same bound but not the same bits
    for pad in (0, 5):
        check(q, cache, table, ptable, groups, [333], own, counts, mask=mask, pad=pad)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("seqs", [3, 60])
def test_unseen_pages_and_poisoned_places(dtype, seqs):
    """Page numbers outside the cache are not seen, in a prefix neither; what lies behind a prefix's end, on its last
    page, reaches nobody; a sequence that sees nothing at all is 0."""
    H, D, page, prefix = 4, 64, 32, 300
    own = [b % 7 for b in range(seqs)]
    cache, table, ptable, groups = batch([seqs - 1, 1], [prefix, 40], own, [1] * seqs, H, page, D, 450)
    bad = torch.tensor([float("nan"), float("inf"), float("-inf"), 3e38])
    for name in ("ks", "vs"):
        last = cache[name][ptable[0, prefix // page].long()]            # [H][page]
        last[:, prefix % page:] = bad[torch.arange(page - prefix % page) % 4]
        cache[name][ptable[0, prefix // page].long()] = last
    ptable[0, 2], ptable[0, 4] = -1, 10**6
    ptable[1, :] = -1
    table[seqs - 1, :] = -5
    q = randn(seqs, 4 * H, D, seed=452, dtype=dtype)
    got = check(q, cache, table, ptable, groups, [prefix, 40], own, [1] * seqs)
    assert (got[seqs - 1] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("seqs", [4, 50])
@pytest.mark.parametrize("kind", ["prefix_holds_it", "own_holds_it", "flat", "negative"])
def test_where_the_weight_lies(dtype, seqs, kind):
    """The prefix, or the own tokens, hold nearly all of the weight; all alike; a negative scale."""
    H, D, page = 2, 128, 64
    own = [30 + b % 9 for b in range(seqs)]
    cache, table, ptable, groups = batch([seqs], [500], own, [1] * seqs, H, page, D, 460)
    here = torch.zeros(cache["ks"].shape[0], dtype=torch.bool)
    here[ptable.flatten().long()] = True
    if kind == "prefix_holds_it":
        cache["ks"][~here] *= 1e-3
        cache["vs"][~here] *= 30.0
    if kind == "own_holds_it":
        cache["ks"][here] *= 1e-3
        cache["vs"][here] *= 1e-4
    scale = {"flat": 0.0, "negative": -0.15}.get(kind, 0.5)
    q = randn(seqs, 4 * H, D, seed=461, dtype=dtype)
    check(q, cache, table, ptable, groups, [500], own, [1] * seqs, scale=scale)


def test_without_groups_it_is_tree_attention():
    own, counts = [100, 3], [2, 1]
    cache, table, ptable, groups = batch([2], [0], own, counts, 2, 16, 64, 470)
    q = randn(3, 4, 64, seed=471, dtype=torch.bfloat16)
    want = rq.attn_tree(q.to(DEV), dev_cache(cache), table.to(DEV), i32(own).to(DEV), i32([0, 2, 3]).to(DEV), SEED, max_nodes=2)
    got = run(q, cache, table, ptable, groups, [0], own, counts)
    none = run(q, cache, table, torch.zeros(0, 3, dtype=torch.int32), i32([0]), [], own, counts)
    assert torch.equal(got, want) and torch.equal(none, want)


@pytest.mark.parametrize("seqs,dtype", [(3, torch.float32), (64, torch.bfloat16)])
def test_streams_graphs_workspaces_and_repeats(seqs, dtype):
    H, D, page = 4, 128, 64
    own = [(17 * b) % 300 for b in range(seqs)]
    cache, table, ptable, groups = batch([seqs], [2000], own, [1] * seqs, H, page, D, 480)
    rows = randn(seqs, 3 * 4 * H, D, seed=481, dtype=dtype)
    q = rows[:, 4 * H:8 * H]                                        # rows three times as far apart
    want = check(q.contiguous(), cache, table, ptable, groups, [2000], own, [1] * seqs, blocks=True)
    d = lambda x: x.to(DEV)
    dc, dq, args = dev_cache(cache), d(rows)[:, 4 * H:8 * H], (d(table), d(i32(own)), d(i32(range(seqs + 1))), d(ptable), d(i32([2000])), d(groups))
    call = lambda **kw: rq.attn_prefix(dq, dc, *args, SEED, max_nodes=1, **kw)
    for _ in range(5):
        assert torch.equal(call(), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    ws = torch.full((rq.attn_prefix_workspace(seqs, 4 * H, D),), 255, dtype=torch.uint8, device=DEV)      # NaN, should it be read
    assert torch.equal(call(workspace=ws), want)
    with pytest.raises(rq.RQError):
        call(workspace=ws[:-16])
    out = torch.empty_like(want)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph in graphs:                                            # two graphs share one workspace
        with torch.cuda.graph(graph):
            call(workspace=ws, out=out)
    for graph in graphs * 2:
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("seqs,groups,prefix,own,heads,kv_heads,page,hidden", [
    (1, 1, 1, 0, 4, 4, 16, 16),
    (5, 2, 100, 40, 8, 2, 32, 250),
    (40, 1, 2100, 33, 16, 4, 64, 512),
])
def test_steps_in_a_row(seqs, groups, prefix, own, heads, kv_heads, page, hidden):
    """Plan, write, turn, attend, project, several tokens over page ends; then the same steps from a graph."""
    work, again = (PrefixStep(seqs, groups, prefix, own, heads, kv_heads, page, hidden, steps=40) for _ in range(2))
    # bf16: the rows are rounded by 2^-8 at most each on the way out and y once more, queries, keys and values as in
    # tree attention; rounding errors of a row add up as squares, so their share of a row is below 2^-8 each
    for _ in range(20):
        q, _, y = work.step()
    assert work.error(q, y) < 2 * 2.0**-8
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again.step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        _, _, y2 = again.step()
    for _ in range(19):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2, y) and torch.equal(work.table, again.table) and torch.equal(work.head, again.head)


@pytest.mark.parametrize("dtype,seqs,groups,G", [(torch.float32, 100, 100, 1), (torch.bfloat16, 100, 100, 2), (torch.float16, 1360, 40, 1),
                                                 (torch.bfloat16, 1360, 40, 1), (torch.bfloat16, 5200, 40, 1)])
def test_units_of_several_pieces(dtype, seqs, groups, G):
    """More units than blocks, each of more tiles than one accumulator adds up: a unit's pieces go on from one another
    and from the pass before.  Against tree attention over tables that name the prefix for each sequence; all groups
    name the same pages, so that they fit.  Either is off by its roundings: 2^-11 of a weight, twice that where keys and
    values are folded, the queries' (4/3) delta with delta below one here, and the output's."""
    H, D, page, pages = 4, 64, 256, 160                              # 40,960 tokens: 320 tiles
    own = [1 + b % 3 for b in range(seqs)]
    cache = dev_cache(filled_cache(pages + seqs, H, page, D, 490))
    ptable = torch.arange(pages, dtype=torch.int32).repeat(groups, 1)
    table = pages + torch.arange(seqs, dtype=torch.int32)[:, None]
    bounds = i32([seqs * i // groups for i in range(groups + 1)])
    q = randn(seqs, H * G, D, seed=491, dtype=dtype).to(DEV)
    d = lambda x: x.to(DEV)
    ctx, offsets = d(i32(own)), d(i32(range(seqs + 1)))
    got = rq.attn_prefix(q, cache, d(table), ctx, offsets, d(ptable), d(i32([pages * page] * groups)), d(bounds), SEED, max_nodes=1)
    joint = torch.cat([ptable[:1].repeat(seqs, 1), table], 1).contiguous()
    want = rq.attn_tree(q, cache, d(joint), ctx + pages * page, offsets, SEED, max_nodes=1).double()
    part = 2.0**-21 if dtype == torch.float32 else 2.0**-10
    # a row of such an average is short beside the values that it averages: sum p |v| is below 4 sigma sqrt(D) of them
    err, bound = (got.double() - want).norm(dim=-1), 2 * (8e-6 + 2 * part * (7 / 3)) * 4 * D**0.5 + 2 * paged_ref.UNIT[dtype] * want.norm(dim=-1)
    assert torch.isfinite(want).all() and (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes,G", [((2, 1, 3), 4), ((1, 1), 1), ((30, 1, 59), 4), ((300,), 8)])
@pytest.mark.parametrize("fill", [0, 127, 255])
def test_tables_wider_than_the_prefixes(dtype, sizes, G, fill):
    """The launches go by the tables' widths: more blocks than there are tiles, some without any.  Whatever lay in the
    workspace."""
    H, D, page = 2, 64, 16
    seqs = sum(sizes)
    prefixes, own, counts = [(300, 0, 130)[i] for i in range(len(sizes))], [7 * b % 50 for b in range(seqs)], [1] * seqs
    cache, table, ptable, groups = batch(list(sizes), prefixes, own, counts, H, page, D, 500)
    wide = torch.cat([ptable, torch.full((len(sizes), 400), -1, dtype=torch.int32)], 1)
    ws = torch.full((rq.attn_prefix_workspace(seqs, H * G, D),), fill, dtype=torch.uint8, device=DEV)
    q = randn(seqs, H * G, D, seed=501, dtype=dtype)
    got = run(q, cache, table, wide, groups, prefixes, own, counts, workspace=ws)
    assert torch.equal(got, run(q, cache, table, wide, groups, prefixes, own, counts, workspace=ws))
    check(q, cache, table, ptable, groups, prefixes, own, counts)
    check(q, cache, table, wide, groups, prefixes, own, counts, workspace=ws)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("groups,prefix", [(2, 700), (40, 16), (40, 700), (1, 5000)])
def test_blocks_of_many_own_rows(dtype, groups, prefix):
    """Trees of 9 nodes and 4 query heads to a KV head: the second pass takes blocks of 128 rows and more too."""
    H, G, D, n, seqs = 2, 4, 64, 9, 40
    own, counts = [500 + 3 * b for b in range(seqs)], [n] * seqs
    cache, table, ptable, bounds = batch([seqs // groups] * groups, [prefix] * groups, own, counts, H, 16, D, 510)
    q = randn(n * seqs, H * G, D, seed=511, dtype=dtype)
    check(q, cache, table, ptable, bounds, [prefix] * groups, own, counts, mask=paged_ref.tree_mask(counts, gen(512)), blocks=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("before,sizes,after", [(2, (0, 3, 0, 2), 1), (0, (1, 0), 40), (33, (70, 0, 1), 5)])
def test_sequences_of_no_group_and_groups_of_none(dtype, before, sizes, after):
    H, G, D = 2, 4, 64
    seqs = before + sum(sizes) + after
    prefixes, own, counts = [130 + 100 * i for i in range(len(sizes))], [11 * b % 160 for b in range(seqs)], [1 + b % 2 for b in range(seqs)]
    cache, table, ptable, groups = batch(list(sizes), prefixes, own, counts, H, 16, D, 520)
    check(randn(sum(counts), H * G, D, seed=521, dtype=dtype), cache, table, ptable, groups + before, prefixes, own, counts, pad=2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sizes,prefixes,n", [((300,), (700,), 1), ((70, 40, 90), (2500, 0, 129), 1), ((40, 33), (900, 260), 9)])
def test_blocks_of_256_rows(D, sizes, prefixes, n):
    """Tables wide enough for the blocks that long prefixes take; rows that fill the last block in part."""
    H, G, page, seqs = 2, 4, 16, sum(sizes)
    own, counts = [(300 if n > 1 else 0) + 13 * b % 200 for b in range(seqs)], [n] * seqs
    cache, table, ptable, groups = batch(list(sizes), list(prefixes), own, counts, H, page, D, 530)
    wide = torch.cat([ptable, torch.full((len(sizes), 6200), -1, dtype=torch.int32)], 1)
    mask = paged_ref.tree_mask(counts, gen(532)) if n > 1 else None
    check(randn(n * seqs, H * G, D, seed=531, dtype=torch.bfloat16), cache, table, wide, groups, list(prefixes), own, counts,
          mask=mask, blocks=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("seqs,n", [(3, 1), (300, 2), (60, 20)])
@pytest.mark.parametrize("page,wide", [(128, 1), (16, 8), (16, 9)])
def test_tables_of_one_tile(dtype, seqs, n, page, wide):
    """What no sequence can pass is a tile, or one page more; more units than blocks too."""
    H, G, D = 2, 2, 64
    own, counts = [(31 * b) % (128 - n + 1) for b in range(seqs)], [n] * seqs
    cache, table, ptable, groups = batch([seqs], [100], own, counts, H, page, D, 540)
    table = torch.cat([table, torch.full((seqs, max(0, wide - table.shape[1])), -1, dtype=torch.int32)], 1)
    mask = paged_ref.tree_mask(counts, gen(542)) if n > 1 else None
    check(randn(n * seqs, H * G, D, seed=541, dtype=dtype), cache, table, ptable, groups, [100], own, counts, mask=mask, blocks=n > 8)
