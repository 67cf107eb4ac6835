"""Block tables and slots from request lengths: every number equal to the plain form's."""
import numpy as np
import pytest
import torch

import prefix_ref as ref
import rotational_w4a4_quantization_gb300 as rq
from test_gpu_paged import DEV, SEED, _built, _status, gen, randn  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def check(contexts, new, table, free, total, page, head=None, base=None, **kw):
    want = ref.plan(contexts, new, table.tolist(), free, total, page, 0 if head is None else head, base)
    t = table.to(DEV)
    got = rq.kv_plan(i32(contexts), i32(new), t, i32(free), total, page, head=None if head is None else i32([head]),
                     base=None if base is None else i32(base), **kw)
    for g, w, dt in zip(got, want, (torch.int32, torch.int64, torch.int64, torch.int32)):
        assert g.dtype == dt and g.tolist() == (w if isinstance(w, list) else [w])
    assert t.tolist() == want[4]
    return got, t


def case(B, most_ctx, most_new, page, seed, spare=3, width=None):
    g = gen(seed)
    ctx = torch.randint(0, most_ctx + 1, (B,), generator=g).tolist()
    new = torch.randint(0, most_new + 1, (B,), generator=g).tolist()
    need = sum(-(-(c + n) // page) for c, n in zip(ctx, new))
    order = torch.randperm(need + spare, generator=g).tolist()
    W = width or max(1, max((-(-(c + n) // page) for c, n in zip(ctx, new)), default=1) + 1)
    table = torch.full((B, W), 77, dtype=torch.int32)
    for b, c in enumerate(ctx):
        k = min(-(-c // page), W)
        table[b, :k] = torch.tensor(order[:k], dtype=torch.int32)
        order = order[k:]
    return ctx, new, table, order


@pytest.mark.parametrize("B", [1, 2, 31, 511, 512, 513, 1025, 4099])
@pytest.mark.parametrize("most_ctx,most_new,page", [(300, 1, 64), (40, 33, 16), (0, 70, 32)])
def test_requests(B, most_ctx, most_new, page):
    """Numbers of requests around a block's threads; padded rows behind the last token."""
    ctx, new, table, free = case(B, most_ctx, most_new, page, B + most_new)
    check(ctx, new, table, free, sum(new) + 5, page, base=[(7 * b) % 1000 for b in range(B)])


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("c", [0, 1, 15, 16, 17, 255, 256, 257])
@pytest.mark.parametrize("n", [0, 1, 16, 300])
def test_pages_around_their_ends(page, c, n):
    ctx, new, table, free = case(3, 0, 0, page, 1)
    need = -(-(c + n) // page)
    table = torch.arange(3 * (need + 1), dtype=torch.int32).view(3, need + 1)
    check([c, 0, c], [n, 2, n], table, list(range(1000, 1000 + 3 * need + 3)), 2 * n + 2, page, head=2)


def test_few_long_requests():
    ctx, new, table, free = case(3, 5000, 40000, 16, 5)
    check(ctx, new, table, free, sum(new), 16)


@pytest.mark.parametrize("B", [1, 600])
def test_pages_that_are_not_there(B):
    """A free list that ends early or begins past its end, a table that is too narrow, rows that are too few."""
    ctx, new, table, free = case(B, 100, 90, 16, 11)
    check(ctx, new, table, free[:len(free) // 2], sum(new), 16)
    check(ctx, new, table, free, sum(new), 16, head=len(free) - 1)
    check(ctx, new, table, [], sum(new), 16)
    check(ctx, new, table, free, sum(new) // 2, 16)
    check(ctx, new, table, free, 0, 16)
    check(ctx, new, table[:, :2].contiguous(), free, sum(new), 16)
    check(ctx, new, table, free, sum(new), 16, head=-3)
    check([-5 if b % 2 else c for b, c in enumerate(ctx)], [-1 if b % 3 == 0 else n for b, n in enumerate(new)], table, free,
          sum(new), 16)


def test_nothing_to_plan():
    check([], [], torch.zeros(0, 4, dtype=torch.int32), [1, 2], 3, 64, head=1)
    check([], [], torch.zeros(0, 4, dtype=torch.int32), [], 0, 64)
    check([5, 6], [0, 0], torch.zeros(2, 1, dtype=torch.int32), [3], 0, 64)
    check([5, 6], [1, 2], torch.zeros(2, 0, dtype=torch.int32), [3], 3, 64)      # no table: no slots


def test_given_outputs_streams_and_graphs():
    """A captured step whose lengths and head advance on the device gives each step's plan."""
    B, page, steps = 5, 16, 40
    ctx, new, table, free = case(B, 30, 0, page, 21, spare=40, width=8)
    with pytest.raises(ValueError, match="out \\(slots\\)"):
        rq.kv_plan(i32(ctx), i32(new), table.to(DEV), i32(free), 3, page, out=(i32([0] * 6), i32([0] * 3), i32([0] * 3), i32([0])))
    one = [b % 2 + 1 for b in range(B)]
    c, n, t, f, h = i32(ctx), i32(one), table.to(DEV), i32(free), i32([0])
    out = (i32([0] * (B + 1)), torch.zeros(9, dtype=torch.int64, device=DEV), torch.zeros(9, dtype=torch.int64, device=DEV), i32([0]))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step(**kw):
        rq.kv_plan(c, n, t, f, 9, page, head=h, out=out, **kw)
        c.add_(n)
        h.copy_(out[3])

    with torch.cuda.stream(s):
        step()
    s.synchronize()
    c.copy_(i32(ctx)), t.copy_(table), h.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    lens, rows, head = list(ctx), table.tolist(), 0
    for _ in range(steps):
        graph.replay()
        torch.cuda.synchronize()
        offsets, slots, positions, head, rows = ref.plan(lens, one, rows, free, 9, page, head)
        assert [x.tolist() for x in out] == [offsets, slots, positions, [head]] and t.tolist() == rows
        lens = [a + b for a, b in zip(lens, one)]
    got = rq.kv_plan(i32(ctx), i32(one), table.to(DEV), f, 9, page, stream=s)
    s.synchronize()
    assert got[1].tolist() == ref.plan(ctx, one, table.tolist(), free, 9, page)[1]


def test_slots_are_what_append_and_read_take():
    """Prompts written by their plan read back as they were, whatever pages they got."""
    H, D, page, B = 2, 64, 16, 7
    ctx, new, table, free = case(B, 0, 50, page, 31)
    total = sum(new)
    (off, slots, pos, _), t = check([0] * B, new, table, free, total + 3, page)
    k = randn(total + 3, H, D, seed=32).to(DEV)
    cache = rq.kv_cache(max(free) + 1, H, D, page)
    rq.kv_append(k, k, cache, slots, SEED)
    got, _ = rq.kv_read(cache, t, None, off, total, SEED, dtype=torch.float32)
    plain = rq.kv_cache(-(-(total + 3) // page), H, D, page)
    rq.kv_append(k, k, plain, torch.arange(total + 3, device=DEV), SEED)
    want, _ = rq.kv_read(plain, torch.arange(plain["kq"].shape[0], dtype=torch.int32, device=DEV)[None], None, i32([0, total]),
                         total, SEED, dtype=torch.float32)
    assert torch.equal(got, want) and np.isfinite(got.cpu().numpy()).all()
