"""Block tables and slots of as many requests as a call takes, against the plain form's numbers."""
import pytest

from test_gpu_paged import _built, _status  # noqa: F401
from test_gpu_plan import case, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,most_ctx,most_new,page", [(65536, 90, 1, 32), (65535, 40, 3, 16), (20000, 0, 20, 16)])
def test_many_requests(B, most_ctx, most_new, page):
    """Stretches of up to 128 requests to a thread; a free list that ends before the last of them; padded rows."""
    ctx, new, table, free = case(B, most_ctx, most_new, page, B, spare=0)
    check(ctx, new, table, free[:-5], sum(new) + 7, page, base=[b % 1000 for b in range(B)])
