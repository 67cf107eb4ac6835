"""Shared-prefix attention where its two passes take unlike blocks."""
import pytest
import torch

import paged_ref
from test_gpu_paged import _built, _status, gen, randn  # noqa: F401
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
