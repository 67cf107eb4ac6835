"""Shared-prefix attention where its two passes take unlike blocks, and where units go on in several pieces: each tile of
the prefix has a place of its own in the result, so that one that is lost or counted twice cannot hide."""
import pytest
import torch

import paged_ref
import rotational_w4a4_quantization_gb300 as rq
from test_gpu_paged import DEV, SEED, _built, _status, dev_cache, filled_cache, gen, randn  # noqa: F401
from test_gpu_prefix import batch, check

pytestmark = pytest.mark.gpu


def tiles(rows, most, groups, H, G, block, width, page):
    """The tiles by which the library chooses its kernels: as many as the table can name."""
    return H * min(groups * -(-most * G // block), groups + rows * G // block) * -(-width * page // 128)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefixes,sizes", [((600,), (40,)), ((300, 0, 129), (38, 1, 1))])
def test_few_rows_before_many(dtype, D, prefixes, sizes):
    """The prefix on blocks of 16 rows, over several of them, the own tokens on those of 128 and more: the join between
    the passes leaves every row in the state."""
    H, G, n, page, seqs = 2, 4, 9, 16, 40
    own, counts = [480 + b % 24 for b in range(seqs)], [n] * seqs
    cache, table, ptable, groups = batch(list(sizes), list(prefixes), own, counts, H, page, D, 700)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = n * seqs
    assert tiles(rows, rows, len(sizes), H, G, 128, ptable.shape[1], page) <= sms < tiles(rows, n, seqs, H, G, 128, table.shape[1], page)
    assert ptable.shape[1] * page > 128 and n * G > 32               # so there is a join, and the second pass is not of few rows
    q = randn(rows, H * G, D, seed=701, dtype=dtype)
    check(q, cache, table, ptable, groups, list(prefixes), own, counts, mask=paged_ref.tree_mask(counts, gen(702)), blocks=True)


@pytest.mark.parametrize("dtype,seqs,groups,G", [(torch.float32, 100, 100, 1), (torch.bfloat16, 100, 100, 2), (torch.float16, 1360, 40, 1),
                                                 (torch.bfloat16, 1360, 40, 1), (torch.bfloat16, 5200, 40, 1)])
def test_every_tile_of_every_piece(dtype, seqs, groups, G):
    """More units than blocks, each of 320 tiles in two pieces.  A token's value is 7 of its scale at dim `tile % 64` and 0
    elsewhere, own tokens have all dims, and the rows stay in the rotated basis: an element is a sum of five tiles and the
    own tokens, all positive, so that its relative error is at most that of its terms and of the sum of the weights:
      scores: q~ and, folded, the keys rounded by u each (2^-11, fp32 2^-22): 2 u S with S = scale sum |q~ k|, in both sums;
      weights by u in both, folded values by u;
      additions: 2^-23 of the sum at most for each of 256 x 8, 2^-12;   the result's own rounding."""
    H, D, page, pages, T = 4, 64, 256, 160, 320
    own = [1 + b % 3 for b in range(seqs)]
    cache = filled_cache(pages + seqs, H, page, D, 710)
    cache["vq"][:pages] = 0
    for t in range(T):
        dim = t % D
        cache["vq"][t // 2, :, 128 * (t & 1):128 * (t & 1) + 128, dim // 2] = 7 << (4 * (dim & 1))
    cache["vq"][pages:] = 0x55
    cache["vs"][pages:] = 30.0
    cache = dev_cache(cache)
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).to(DEV)
    ptable = torch.arange(pages, dtype=torch.int32).repeat(groups, 1).to(DEV)
    table = (pages + torch.arange(seqs, dtype=torch.int32))[:, None].to(DEV)
    q = randn(seqs, H * G, D, seed=711, dtype=dtype).to(DEV)
    turned = (q.double() @ paged_ref.rotation(D, SEED, 1).to(DEV)).view(seqs, H, G, D)
    there = torch.arange(page, device=DEV)[None, :] <= i32(own)[:, None]                   # own tokens and the node

    def rows(h):
        """Of a KV head: keys and value scales of the prefix, keys of the sequences' own pages."""
        k = paged_ref.decode(cache["kq"][:, h, :], cache["ks"][:, h, :])
        return k[:pages].flatten(0, 1), cache["vs"][:pages, h].double().flatten(), k[pages:]

    def chunks():
        for h in range(H):
            k, vs, ko = rows(h)
            for a in range(0, seqs, 256):
                yield h, a, turned[a:a + 256, h].flatten(0, 1), k, vs, ko[a:a + 256, :8].repeat_interleave(G, 0), there[a:a + 256, :8].repeat_interleave(G, 0)

    most = 0.0                                                        # sum |q~ k| over all that is seen
    for h, a, x, k, vs, ko, see in chunks():
        most = max(most, float((x.abs() @ k.abs().T).max()), float(torch.einsum("nd,ntd->nt", x.abs(), ko.abs())[see].max()))
    S = 4.0
    scale = S / most
    bounds = i32([seqs * i // groups for i in range(groups + 1)])
    got = rq.attn_prefix(q, cache, table, i32(own), i32(range(seqs + 1)), ptable, i32([pages * page] * groups), bounds, SEED,
                         rq.RQ_SIGNS_FIRST | rq.RQ_ATTN_ROTATED_OUT, max_nodes=1, softmax_scale=scale).double().view(seqs, H, G, D)
    u = 2.0**-22 if dtype == torch.float32 else 2.0**-11
    bound = 4 * u * S + 3 * u + 2.0**-12 + paged_ref.UNIT[dtype]
    for h, a, x, k, vs, ko, see in chunks():
        w = torch.exp(x @ k.T * scale)
        tile = (w * vs * 7).view(-1, T, 128).sum(-1)
        wo = torch.where(see, torch.exp(torch.einsum("nd,ntd->nt", x, ko) * scale), 0.0)
        mine = wo.sum(-1, keepdim=True) * 5 * 30.0
        total = tile.view(-1, T // D, D).sum(1) + mine
        want = total / (w.sum(-1) + wo.sum(-1))[:, None]
        # what a lost tile, or lost own tokens, would change stands well above the bound
        assert float((tile.view(-1, T // D, D) / total[:, None]).min()) > 3 * bound and float((mine / total).min()) > 3 * bound
        err = ((got[a:a + 256, h].flatten(0, 1) - want).abs() / want).max()
        assert err <= bound, float(err / bound)
