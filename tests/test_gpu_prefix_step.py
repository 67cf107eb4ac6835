"""Decode steps of more requests than a product with 4-bit weights takes rows."""
import pytest
import torch

from rotational_w4a4_quantization_gb300.prefix_step import PrefixStep
from test_gpu_paged import _built, _status  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs,groups,hidden", [(64, 1, 250), (65, 2, 250), (130, 3, 128)])
def test_more_requests_than_rows_of_a_product(seqs, groups, hidden):
    """Against 64 bits: the attention's rows and their projection are each rounded to bf16, 2^-8 of a value at most;
    roundings of a row add up as squares, so their share of a row is below 2^-8 each."""
    work = PrefixStep(seqs, groups, 300, 40, 8, 2, 32, hidden, steps=4)
    work.y.fill_(float("nan"))
    for _ in range(2):
        q, _, y = work.step()
    assert torch.isfinite(y).all() and work.error(q, y) < 2 * 2.0**-8
