"""Calls of the rotary, paged-cache and tree entry points as users make them: gradients through rope, strides of
dimensions of size one, a mask shared by all nodes, contexts far past the table, workspaces, values near fp32's end."""
import math

import numpy as np
import pytest
import torch

import paged_ref as ref
import rotational_w4a4_quantization_gb300 as rq
from test_gpu_paged import DEV, DTYPES, SEED, _built, _status, check_tree, dev_cache, gen, paged, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [32, 64, 128, 256])
def test_workspace_is_that_of_the_kernels_that_run(D):
    """Heads of 32 and 256 elements have no blocks of 128 rows: two partials of 16 rows a block, three blocks to an SM."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    few = 2 * 3 * sms * 16 * (D + 2) * 4 + 64 * 4 * sms
    many = 2 * sms * 256 * (D + 2) * 4 + 64 * sms
    assert 0 < rq.attn_tree_workspace(D) <= (few if D in (32, 256) else max(few, many))


@pytest.mark.parametrize("n", [1, 40])
def test_contexts_far_past_the_table(n):
    """What lies past the table is not seen, also where the number of tokens is int32's last."""
    H, D, page = 2, 64, 16
    cache, table = paged([200] * 60, H, page, D, 600)
    q = randn(60 * n, 4 * H, D, seed=601, dtype=torch.bfloat16)
    a, b = (check_tree(q, cache, table, [c] * 60, [n] * 60) for c in (table.shape[1] * page, 2**31 - 1))
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("G,n", [(4, 3), (4, 12)])
def test_one_mask_row_for_all_nodes(dtype, G, n):
    B, H, D = 50, 2, 64
    contexts, counts = [150 + b for b in range(B)], [n] * B
    cache, table = paged([c + n for c in contexts], H, 32, D, 610)
    one = torch.zeros(1, n, dtype=torch.bool)
    one[0, ::2] = True
    q = randn(B * n, H * G, D, seed=611, dtype=dtype)
    want = check_tree(q, cache, table, contexts, counts, mask=one.repeat(B * n, 1))
    offsets = torch.arange(0, B * n + 1, n, dtype=torch.int32, device=DEV)
    got = rq.attn_tree(q.to(DEV), dev_cache(cache), table.to(DEV), torch.tensor(contexts, dtype=torch.int32, device=DEV),
                       offsets, SEED, 1, tree_mask=one.to(DEV).expand(B * n, n))
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_strides_of_dimensions_of_size_one(dtype):
    """One token whose row is an odd slice, one head at an odd stride: strides that nothing uses are not asked of."""
    D, page = 64, 16
    rows = randn(3, 3 * D + 5, seed=620, dtype=dtype).to(DEV)
    odd = lambda x: x.as_strided(x.shape, [s if n > 1 else s + 5 for n, s in zip(x.shape[:2], x.stride()[:2])] + [1])
    k1, v1 = (rows[0, i * D:(i + 1) * D].view(1, 1, D) for i in (0, 1))
    cache, plain = rq.kv_cache(2, 1, D, page), rq.kv_cache(2, 1, D, page)
    slot = torch.tensor([5], device=DEV)
    rq.kv_append(odd(k1), odd(v1), cache, slot, SEED)
    rq.kv_append(k1.contiguous(), v1.contiguous(), plain, slot, SEED)
    assert all(torch.equal(cache[x], plain[x]) for x in cache)
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    got = rq.attn_tree(odd(k1), cache, table, i32(6), i32(0, 1), SEED)
    assert torch.equal(got, rq.attn_tree(k1.contiguous(), cache, table, i32(6), i32(0, 1), SEED))
    turns, _ = rq.rope_turns(D)
    pos = torch.tensor([77], device=DEV)
    for a, b in zip(rq.rope(odd(k1), odd(v1), pos, turns), rq.rope(k1.contiguous(), v1.contiguous(), pos, turns)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("who", ["qk", "q", "k"])
def test_rope_carries_gradients(interleaved, dtype, who):
    """backward() through rope: the transposed turn of what comes back, for q, k or both; also where the gradient that
    arrives is a broadcast value, and where it passes a slice of a projection's rows."""
    T, H, K, D, rot = 9, 4, 2, 64, 48
    turns, m = rq.rope_turns(rot, scaling="parts", factor=4.0)
    pos = torch.randint(0, 9000, (T,), generator=gen(630)).to(DEV)
    rows = randn(T, (H + K) * D, seed=631, dtype=dtype).to(DEV)
    rows.requires_grad_()
    parts = {"q": rows[:, :H * D].view(T, H, D), "k": rows[:, H * D:].view(T, K, D)}
    q, k = (parts[n] if n in who else parts[n].detach() for n in "qk")
    q2, k2 = rq.rope(q, k, pos, turns, interleaved=interleaved, mscale=m)
    assert q2.requires_grad == ("q" in who) and k2.requires_grad == ("k" in who)
    gq, gk = (randn(T, n, D, seed=632 + n, dtype=dtype).to(DEV) for n in (H, K))
    loss = 0.0
    if "q" in who:
        loss = loss + (q2 * gq).sum()
    if "k" in who:
        loss = loss + (k2 * gk).sum() + k2[..., rot:].sum() * 0
    loss.backward()
    back = rq.rope(gq, gk, pos, turns, interleaved=interleaved, inverse=True, mscale=m)
    want = torch.zeros_like(rows)
    if "q" in who:
        want[:, :H * D] = back[0].view(T, -1)
    if "k" in who:
        want[:, H * D:] = back[1].view(T, -1)
    assert torch.equal(rows.grad, want)
    rows.grad = None
    y = rq.rope(rows[:, :H * D].view(T, H, D), None, pos, turns, interleaved=interleaved, mscale=m)[0]
    y.sum().backward()                                           # the gradient of a sum has strides of 0
    one = rq.rope(torch.ones(T, H, D, dtype=dtype, device=DEV), None, pos, turns, interleaved=interleaved, inverse=True, mscale=m)[0]
    assert torch.equal(rows.grad[:, :H * D], one.view(T, -1)) and (rows.grad[:, H * D:] == 0).all()


def test_rope_gradient_by_differences():
    """And against differences of the formula in 64 bits."""
    T, H, D = 3, 2, 32
    turns, _ = rq.rope_turns(D, device="cpu")
    pos = torch.tensor([0, 5, 131071])
    x = randn(T, H, D, seed=640).to(DEV).requires_grad_()
    g = randn(T, H, D, seed=641).to(DEV)
    y, _ = rq.rope(x, None, pos.to(DEV), turns.to(DEV))
    y.backward(g)
    x64, g64 = x.detach().cpu().double(), g.cpu().double()
    for t, h, d in [(0, 0, 0), (1, 1, 7), (2, 0, 31), (2, 1, 16)]:
        e = torch.zeros(T, H, D, dtype=torch.float64)
        e[t, h, d] = 1.0                                         # the turn is linear
        diff = ((ref.turn(x64 + e, pos, turns, False) - ref.turn(x64 - e, pos, turns, False)) * g64).sum() / 2
        assert abs(float(diff) - float(x.grad[t, h, d])) < 2e-6 * float(g.abs().max())


def test_rope_refuses_out_where_gradients_are_asked_for():
    turns, _ = rq.rope_turns(32)
    x, pos = torch.zeros(2, 1, 32, device=DEV, requires_grad=True), torch.zeros(2, dtype=torch.int64, device=DEV)
    with pytest.raises(ValueError, match="gradients"):
        rq.rope(x, None, pos, turns, out=(torch.empty(2, 1, 32, device=DEV), None))
    with torch.no_grad():
        assert not rq.rope(x, None, pos, turns, out=(torch.empty(2, 1, 32, device=DEV), None))[0].requires_grad


def test_rotary_coefficients():
    """cos and sin of an angle that is exact modulo a turn: folded to an eighth of a turn, its fp32 form is off by at
    most 2^-25 of pi/4 (2.4e-8), and sincospif by one ulp of its result."""
    D, T = 256, 4096
    g = gen(650)
    turns = torch.randint(-2**62, 2**62, (D // 2,), generator=g)
    pos = torch.randint(0, 2**40, (T,), generator=g)
    x = torch.zeros(T, 1, D)
    x[..., :D // 2] = 1.0
    y, _ = rq.rope(x.to(DEV), None, pos.to(DEV), turns.to(DEV))
    p, w = pos.numpy().astype(np.uint64)[:, None], turns.numpy().astype(np.uint64)[None, :]
    phase = p * w                                                # wraps modulo one turn
    whole = phase >> np.uint64(61)                               # eighths, so that the rest keeps 53 bits
    rest = (phase & np.uint64(2**61 - 1)).astype(np.float64) * (2 * math.pi * 2.0**-64)
    eighth = whole.astype(np.float64) * (math.pi / 4)
    cos = np.cos(eighth) * np.cos(rest) - np.sin(eighth) * np.sin(rest)
    sin = np.sin(eighth) * np.cos(rest) + np.cos(eighth) * np.sin(rest)
    got = y[:, 0].cpu().double().numpy()
    ulp = lambda v: np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 1e-12))) - 23)
    for have, want, other in ((got[:, :D // 2], cos, sin), (got[:, D // 2:], sin, cos)):
        err = np.abs(have - want)
        assert (err <= 2.4e-8 * np.abs(other) + ulp(want) + 1e-15).all(), float((err - 2.4e-8 * np.abs(other) - ulp(want)).max())


def test_append_rows_near_the_end_of_fp32():
    """A finite row whose sums pass fp32's range before they are divided by sqrt(D) has scale NaN, as one that holds an
    infinity; a row whose sums stay inside is kept."""
    H, D, page = 1, 64, 16
    k = torch.full((4, H, D), 1e38)
    k[1] = 3e38 / D / 2
    k[2] = torch.where(torch.arange(D) % 2 == 0, 3e38, -3e38)
    cache = rq.kv_cache(1, H, D, page)
    rq.kv_append(k.to(DEV), k.to(DEV), cache, torch.arange(4, device=DEV), SEED, 1)
    for n in "kv":
        s = cache[n + "s"][0, 0, :4].cpu()
        assert torch.isnan(s[[0, 2, 3]]).all() and torch.isfinite(s[1])
