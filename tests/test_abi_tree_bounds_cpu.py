"""Host-side checks of tree attention on sizes whose products pass 64 bits."""

import pytest

from test_abi_paged_cpu import lib, tree  # noqa: F401


@pytest.mark.parametrize("kw", [
    dict(nodes=1 << 62),                      # times 32 query heads: 2^67
    dict(nodes=1 << 31),
    dict(nodes=1 << 59),
    dict(W=1 << 60),                          # times 64 rows to a page: 2^66
    dict(W=1 << 58),
])
def test_products_past_64_bits_are_refused(lib, kw):
    assert tree(lib, **kw) == 2
