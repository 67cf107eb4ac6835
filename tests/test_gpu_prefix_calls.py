"""Calls of shared-prefix attention as a server makes them beside the plain decode step."""
import pytest
import torch

import paged_ref
import prefix_ref as ref
import rotational_w4a4_quantization_gb300 as rq
from test_gpu_paged import DEV, DTYPES, SEED, _built, _status, dev_cache, gen, randn  # noqa: F401
from test_gpu_prefix import batch, check, i32, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("counts,own", [((300,), (0,)), ((130, 1, 257, 64), (0, 40, 9, 128))])
def test_prompts_behind_a_shared_prefix(dtype, D, counts, own):
    """As many new tokens as a prompt has, each of which sees those before it; a token of another request among them."""
    cache, table, ptable, groups = batch([len(counts)], [700], list(own), list(counts), 2, 32, D, 800)
    check(randn(sum(counts), 8, D, seed=801, dtype=dtype), cache, table, ptable, groups, [700], list(own), list(counts), blocks=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("seqs", [3, 40])
def test_more_nodes_than_the_bound(dtype, seqs):
    """Nodes past max_nodes are not there: their rows stay as they are, the others are those of a call without them."""
    H, D, n, most = 2, 64, 7, 4
    own = [5 + 3 * b for b in range(seqs)]
    cache, table, ptable, groups = batch([seqs], [400], own, [n] * seqs, H, 16, D, 810)
    q = randn(seqs * n, 4 * H, D, seed=811, dtype=dtype)
    out = torch.full(q.shape, 3.0, dtype=dtype, device=DEV)
    run(q, cache, table, ptable, groups, [400], own, [n] * seqs, max_nodes=most, out=out)
    rows = out.cpu().view(seqs, n, 4 * H, D)
    assert (rows[:, most:] == 3.0).all()
    few = q.view(seqs, n, 4 * H, D)[:, :most].reshape(-1, 4 * H, D).contiguous()
    want, spread, delta = paged_ref.attention(few, *ref.joined(cache, table, own, [most] * seqs, ptable, [400], groups),
                                              i32([most * b for b in range(seqs + 1)]), SEED, 1, D ** -0.5)
    part = 2.0**-22 if dtype == torch.float32 else 2.0**-12
    folded = 2 if dtype == torch.bfloat16 and seqs * n * 4 > 32 else 1
    err = (rows[:, :most].reshape(want.shape).double() - want).norm(dim=-1)
    bound = ((8e-6 + folded * (2 * part + 2 * (4 / 3) * part * delta)) * spread.norm(dim=-1)
             + paged_ref.UNIT[dtype] * want.norm(dim=-1) + (2.0**-25 * D**0.5 if dtype == torch.float16 else 0))
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("seqs", [3, 60, 150])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_that_are_not_finite(dtype, seqs, bad):
    """A query that is not finite reaches its own row and head alone."""
    H, D = 2, 64
    own = [9 + b % 30 for b in range(seqs)]
    cache, table, ptable, groups = batch([seqs], [500], own, [1] * seqs, H, 16, D, 820)
    q = randn(seqs, 4 * H, D, seed=821, dtype=dtype)
    clean = run(q, cache, table, ptable, groups, [500], own, [1] * seqs)
    q[1, 3, 7] = bad
    got = run(q, cache, table, ptable, groups, [500], own, [1] * seqs)
    keep = torch.ones(seqs, 4 * H, dtype=torch.bool)
    keep[1, 3] = False
    assert torch.equal(got[keep.to(DEV)], clean[keep.to(DEV)])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_before_the_first_sequence(dtype):
    """Rows of no sequence at the front, as the rest of a packed batch."""
    H, D, seqs, front = 2, 64, 30, 5
    own = [9 + b % 30 for b in range(seqs)]
    cache, table, ptable, groups = batch([seqs], [500], own, [1] * seqs, H, 16, D, 830)
    q = randn(seqs + front, 4 * H, D, seed=831, dtype=dtype)
    want = check(q[front:], cache, table, ptable, groups, [500], own, [1] * seqs)
    d = lambda x: x.to(DEV)
    out = torch.full(q.shape, 3.0, dtype=dtype, device=DEV)
    rq.attn_prefix(d(q), dev_cache(cache), d(table), d(i32(own)), d(i32(range(front, front + seqs + 1))), d(ptable), d(i32([500])),
                   d(groups), SEED, max_nodes=1, out=out)
    assert (out[:front] == 3.0).all()
    part = 2.0**-10 if dtype == torch.bfloat16 else 1e-5                 # other blocks, other order of the sums
    assert torch.allclose(out[front:].double(), want.double(), rtol=2.0**-7 if dtype == torch.bfloat16 else 1e-4, atol=part)


def test_two_calls_at_once():
    """Two streams, other groups and sizes in each, scratch of their own."""
    H, D = 4, 128
    calls, wants = [], []
    for seqs, prefix, dtype in ((64, 3000, torch.bfloat16), (24, 5000, torch.float16)):
        own = [(17 * b) % 300 for b in range(seqs)]
        cache, table, ptable, groups = batch([seqs], [prefix], own, [1] * seqs, H, 64, D, 840 + seqs)
        args = [x.to(DEV) for x in (table, i32(own), i32(range(seqs + 1)), ptable, i32([prefix]), groups)]
        q, cache = randn(seqs, 4 * H, D, seed=841, dtype=dtype).to(DEV), dev_cache(cache)
        calls.append(lambda stream=None, q=q, cache=cache, args=args: rq.attn_prefix(q, cache, *args, SEED, max_nodes=1, stream=stream))
        wants.append(calls[-1]())
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[call(stream=s) for call, s in zip(calls, streams)] for _ in range(30)]
    torch.cuda.synchronize()
    for pair in got:
        for g, w in zip(pair, wants):
            assert torch.equal(g, w)
