"""Rotary positions, the paged rotated INT4 cache and tree attention against plain
64-bit forms.

Tolerances, derived from the arithmetic:
* rope: a coefficient is off by at most 2.5e-7 (the angle's conversion to fp32, at most
  2^-25 half turns, and one ulp of sin/cos), the two products and their sum by three
  roundings: 1e-6 of the pair's length in all, plus the rounding to the output type.
* cache writes: the fp32 rotation decides the rounding; codes may differ by one only
  where y/scale is within the tie window of a half-integer, scales within 1e-5.
* cache reads: sums of codes are exact, two fp32 roundings of the factor and one of the
  product: 4e-7 relative, plus the rounding to the output type.
* attention: weights are rounded to fp16 (2^-11 of each, 2^-21 in two parts), which is
  at most that much of sum p |v|; rounding the rotated query (2^-12, 2^-22 in two
  parts, independent per element) moves a score by delta = 2^-12 scale sqrt(sum q^2 k^2)
  (one sigma is a third of that; four sigma are allowed for) and so a weight by twice
  that; fp32 scores of up to 45 and the exponential by 8e-6 of a weight.
"""
import numpy as np
import pytest
import torch

import oracle
import paged_ref as ref
import rotational_w4a4_quantization_gb300 as rq
from parity import compare_codes, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
SEED = 0x5EED
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(autouse=True)
def _status():
    yield
    assert rq.sync_status() == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(*shape, seed, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=gen(seed), dtype=torch.float64) * scale).to(dtype)


# ------------------------------------------------------------------ rope

def rope_bound(y, x, rot, interleaved, dtype, mscale):
    """Elementwise: 1e-6 of the pair's length and the output rounding."""
    x = x.double()
    pair = torch.zeros_like(x)
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    length = (a * a + b * b).sqrt() * mscale
    if interleaved:
        pair[..., 0:rot:2] = length
        pair[..., 1:rot:2] = length
    else:
        pair[..., :rot // 2] = length
        pair[..., rot // 2:rot] = length
    u = 0.0 if dtype == torch.float32 else ref.UNIT[dtype] * 1.02
    return 1e-6 * pair + u * y.abs() + (2.0**-25 if dtype == torch.float16 else 0.0)


def check_rope(q, k, pos, turns, interleaved, mscale=1.0, inverse=False, out=None):
    kw = dict(interleaved=interleaved, mscale=mscale, inverse=inverse)
    wants = [None if x is None else ref.turn(x.cpu(), pos, turns, interleaved, mscale, inverse) for x in (q, k)]
    ins = [None if x is None else x.cpu().clone() for x in (q, k)]
    got = rq.rope(q, k, pos.to(DEV), turns.to(DEV), out=out, **kw)
    for x, w, g in zip(ins, wants, got):
        if w is None:
            assert g is None
            continue
        assert g.shape == x.shape and g.dtype == x.dtype
        err = (g.cpu().double() - w).abs()
        assert (err <= rope_bound(w, x, 2 * len(turns), interleaved, x.dtype, mscale)).all(), float(err.max())
    return got


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (64, 48), (96, 72), (256, 192), (64, 2), (10, 6), (256, 256)])
def test_rope_layouts(dtype, interleaved, D, rot):
    """Whole and part of the head; sizes whose pieces are 16 bytes and sizes that go element by element."""
    T = 37
    turns, m = rq.rope_turns(rot, scaling="parts", factor=8.0, device="cpu")
    pos = torch.randint(0, 131072, (T,), generator=gen(1))
    check_rope(randn(T, 6, D, seed=2, dtype=dtype).to(DEV), randn(T, 2, D, seed=3, dtype=dtype).to(DEV), pos, turns,
               interleaved, m)


@pytest.mark.parametrize("T", [0, 1, 2, 255, 4099])
def test_rope_lengths(T):
    turns, _ = rq.rope_turns(128, device="cpu")
    pos = torch.arange(T) + 1000
    check_rope(randn(T, 4, 128, seed=4, dtype=torch.bfloat16).to(DEV), randn(T, 1, 128, seed=5, dtype=torch.bfloat16).to(DEV),
               pos, turns, False)


def test_rope_positions_far_out_and_negative():
    """The angle is exact modulo a turn for every position."""
    turns, _ = rq.rope_turns(64, device="cpu")
    pos = torch.tensor([0, 1, -1, 2**20 + 1, 2**31 + 7, 2**40 + 3, 2**62, -(2**50)])
    check_rope(randn(8, 2, 64, seed=6).to(DEV), None, pos, turns, False)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rope_strides_in_place_and_absent(dtype):
    """Slices of one projection's rows, in place; a transposed head order; rows off the 16-byte grid; q or k alone."""
    T, H, K, D = 19, 4, 2, 64
    turns, _ = rq.rope_turns(D, device="cpu")
    pos = torch.arange(T) * 3
    qkv = randn(T, (H + 2 * K) * D, seed=7, dtype=dtype).to(DEV)
    keep = qkv.clone()
    q, k = qkv[:, :H * D].view(T, H, D), qkv[:, H * D:(H + K) * D].view(T, K, D)
    check_rope(q, k, pos, turns, False)
    assert torch.equal(qkv, keep)                                # out of place: untouched
    check_rope(q, k, pos, turns, True, out=(q, k))
    assert torch.equal(qkv[:, (H + K) * D:], keep[:, (H + K) * D:])
    hm = randn(H, T, D, seed=8, dtype=dtype).to(DEV).transpose(0, 1)
    check_rope(hm, None, pos, turns, False)
    odd = randn(T * H * D + 1, seed=9, dtype=dtype).to(DEV)[1:].view(T, H, D)
    check_rope(None, odd, pos, turns, False)
    odd = randn(T, H, D + 3, seed=10, dtype=dtype).to(DEV)[:, :, :D]
    check_rope(odd, None, pos, turns, True)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(interleaved):
    """The transposed turn is the gradient: of the formula (autograd in 64 bits), and by differences of the kernel."""
    T, H, D, rot = 11, 3, 64, 48
    turns, m = rq.rope_turns(rot, scaling="parts", factor=4.0, device="cpu")
    pos = torch.randint(0, 5000, (T,), generator=gen(11))
    x, g = randn(T, H, D, seed=12), randn(T, H, D, seed=13)
    xd = x.double().requires_grad_()
    w = [int(t) % (1 << 64) for t in turns.tolist()]
    ang = torch.tensor([[((int(p) * f) % (1 << 64)) / 2.0**64 for f in w] for p in pos.tolist()], dtype=torch.float64) * 2 * np.pi
    c, s = (ang.cos() * m)[:, None], (ang.sin() * m)[:, None]
    a, b = (xd[..., 0:rot:2], xd[..., 1:rot:2]) if interleaved else (xd[..., :rot // 2], xd[..., rot // 2:rot])
    turned = torch.cat([a * c - b * s, a * s + b * c, xd[..., rot:]], -1)
    gd = g.double()
    ga, gb = (gd[..., 0:rot:2], gd[..., 1:rot:2]) if interleaved else (gd[..., :rot // 2], gd[..., rot // 2:rot])
    (turned * torch.cat([ga, gb, gd[..., rot:]], -1)).sum().backward()
    got, _ = check_rope(g.to(DEV), None, pos, turns, interleaved, m, inverse=True)
    assert (got.cpu().double() - xd.grad).abs().max() < 2e-6 * float(g.abs().max()) * m * 1.5
    # differences: <g, f(x + h e) - f(x - h e)> / 2h; f is linear, so h is large and the fp32 rounding small
    f = lambda z: rq.rope(z.to(DEV), None, pos.to(DEV), turns.to(DEV), interleaved=interleaved, mscale=m)[0].cpu().double()
    for t, h, d in [(0, 0, 0), (3, 1, 20), (10, 2, 47), (5, 0, 60)]:
        e = torch.zeros(T, H, D)
        e[t, h, d] = 64.0
        diff = float((gd * (f(x + e) - f(x - e))).sum() / 128.0)
        assert abs(diff - float(got[t, h, d])) < 1e-5 * float(g.abs().max())


def test_rope_turns_scalings():
    import math
    for scaling, factor in [("none", 1.0), ("linear", 4.0), ("base", 8.0), ("parts", 16.0), ("smooth", 8.0)]:
        turns, m = rq.rope_turns(64, 10000.0, scaling=scaling, factor=factor, original_length=4096, device="cpu")
        w = torch.tensor([(int(t) % (1 << 64)) / 2.0**64 for t in turns.tolist()], dtype=torch.float64) * 2 * math.pi
        base = 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
        if scaling == "none":
            torch.testing.assert_close(w, base, rtol=1e-12, atol=1e-15)
        if scaling == "linear":
            torch.testing.assert_close(w, base / 4, rtol=1e-12, atol=1e-15)
        if scaling in ("base", "parts", "smooth"):
            assert abs(float(w[0]) - 1.0) < 1e-12                                  # the fastest pair stays
            assert abs(float(w[-1] / base[-1]) * factor - 1.0) < 1e-6              # the slowest is interpolated
        assert m == (0.1 * math.log(16.0) + 1 if scaling == "parts" else 1.0)


# ------------------------------------------------------------------ the paged cache

def filled_cache(pages, H, page, D, seed, scale=1.0):
    """A cache full of codes and scales that no test writes, to see what stays."""
    g = gen(seed)
    c = {}
    for n in "kv":
        c[n + "q"] = torch.randint(0, 256, (pages, H, page, D // 2), generator=g).to(torch.uint8)
        c[n + "s"] = (torch.rand(pages, H, page, generator=g) * 0.4 + 0.05) * scale
    return c


def dev_cache(c):
    return {n: t.to(DEV) for n, t in c.items()}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,page,H", [(32, 16, 3), (64, 32, 8), (128, 64, 2), (256, 128, 1), (128, 16, 5), (128, 256, 8)])
@pytest.mark.parametrize("rope", [None, "half", "interleaved"])
@pytest.mark.parametrize("flags", [0, 1])
def test_append_codes(dtype, D, page, H, rope, flags):
    T, pages = 21, 5
    k, v = randn(T, H, D, seed=20, dtype=dtype), randn(T, H, D, seed=21, dtype=dtype)
    k[:, :, 1] *= 30
    v[:, :, D - 2] *= 30
    slots = torch.randperm(pages * page, generator=gen(22))[:T]
    slots[4], slots[9] = -1, pages * page                     # padding
    before = filled_cache(pages, H, page, D, 23)
    cache = dev_cache(before)
    kw, kr = {}, k.double()
    if rope:
        rot = D // 2 if D >= 64 else D
        turns, m = rq.rope_turns(rot, scaling="parts", factor=2.0, device="cpu")
        pos = torch.randint(0, 100000, (T,), generator=gen(24))
        kw = dict(positions=pos.to(DEV), turns=turns.to(DEV), interleaved=rope == "interleaved", mscale=m)
        kr = ref.turn(k, pos, turns, rope == "interleaved", m)
    assert rq.kv_append(k.to(DEV), v.to(DEV), cache, slots.to(DEV), SEED, flags, **kw) is cache
    keep = torch.ones(pages * page, dtype=torch.bool)
    ok = (slots >= 0) & (slots < pages * page)
    keep[slots[ok]] = False
    pg, row = slots[ok] // page, slots[ok] % page
    for n, x in (("k", kr), ("v", v.double())):
        y = oracle.rotate(x[ok].reshape(-1, D).numpy(), SEED, flags)
        codes, scales, ratio = oracle.quant_rows(y)
        compare_codes(to_np(cache[n + "q"])[pg, :, row].reshape(-1, D // 2), oracle.pack(codes), ratio, D)
        np.testing.assert_allclose(to_np(cache[n + "s"])[pg, :, row].reshape(-1), scales, rtol=1e-5)
        a, b = (c[n + "q"].transpose(1, 2).reshape(pages * page, -1) for c in (before, {n + "q": cache[n + "q"].cpu()}))
        assert torch.equal(a[keep], b[keep])
        a, b = (c[n + "s"].transpose(1, 2).reshape(pages * page, -1) for c in (before, {n + "s": cache[n + "s"].cpu()}))
        assert torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("T", [0, 1, 5, 700])
def test_append_lengths_strides_and_plain_writer(T):
    """Strided views of one projection's rows; without rotary positions the codes are kv_rotate_quant's."""
    H, D, page = 4, 128, 64
    pages = T // page + 2
    rows = randn(max(T, 1), 3 * H * D, seed=30, dtype=torch.bfloat16).to(DEV)[:T]
    k, v = rows[:, H * D:2 * H * D].view(T, H, D), rows[:, 2 * H * D:].view(T, H, D)
    cache = rq.kv_cache(pages, H, D, page)
    slots = torch.arange(T, device=DEV) + 3
    rq.kv_append(k, v, cache, slots, SEED, 1)
    if T:
        want = rq.kv_rotate_quant(k.contiguous(), v.contiguous(), SEED, 1)
        for n in "kv":
            got_s = cache[n + "s"].transpose(1, 2).reshape(pages * page, H)[3:3 + T]
            torch.testing.assert_close(got_s, want[n + "s"], rtol=1e-6, atol=0)
            got_q = cache[n + "q"].transpose(1, 2).reshape(pages * page, H, D // 2)[3:3 + T]
            assert (got_q != want[n + "q"]).float().mean() < 1e-4       # rounding ties alone


def test_append_special_rows():
    """Zero rows keep scale 0; rows with NaN or an infinity get scale NaN and read back as NaN; others are untouched."""
    H, D, page = 2, 64, 16
    k = randn(6, H, D, seed=31)
    v = k.clone()
    k[0] = 0.0
    k[1, 0, 5] = float("nan")
    k[2, 1, 7] = float("inf")
    k[3, 0, 0], k[3, 0, 1] = float("inf"), float("-inf")
    k[4] = 3e38
    k[5] *= 1e-39 / 4
    cache = rq.kv_cache(1, H, D, page)
    rq.kv_append(k.to(DEV), v.to(DEV), cache, torch.arange(6, device=DEV), SEED, 1)
    s = cache["ks"][0].cpu().T                                   # [row][head]
    assert (s[0] == 0).all() and (cache["kq"][0, :, 0] == 0).all()
    for r, h, bad in [(1, 0, True), (1, 1, False), (2, 1, True), (2, 0, False), (3, 0, True), (3, 1, False)]:
        assert bool(torch.isnan(s[r, h])) == bad
    assert torch.isfinite(s[5]).all() and torch.isfinite(cache["vs"][0, :, :6]).all()
    out, _ = rq.kv_read(cache, torch.zeros(1, 1, dtype=torch.int32, device=DEV), None,
                        torch.tensor([0, 6], dtype=torch.int32, device=DEV), 6, SEED, 1, dtype=torch.float32)
    assert torch.isnan(out[1, 0]).all() and torch.isfinite(out[1, 1]).all() and (out[0] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,page,H", [(32, 16, 3), (64, 64, 4), (128, 32, 8), (256, 16, 2)])
@pytest.mark.parametrize("flags", [0, 1, 2, 3])
def test_read(dtype, D, page, H, flags):
    """Ragged ranges, starts inside pages, an empty sequence, page numbers outside the cache, tokens past the table."""
    pages, W = 9, 4
    cache = filled_cache(pages, H, page, D, 40, 1e-3 if dtype == torch.float16 else 3.0)
    table = torch.stack([torch.randperm(pages, generator=gen(41 + b))[:W] for b in range(4)]).to(torch.int32)
    table[2, 1], table[2, 2] = -1, pages
    starts = torch.tensor([0, page + 3, 1, 2 * page], dtype=torch.int32)
    counts = [2 * page + 5, 0, 3 * page, 2 * page + 7]           # the last one runs past its table
    offsets = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)
    total = int(offsets[-1]) + 3                                 # rows past the last sequence stay
    out = tuple(torch.full((total, H, D), 7.0, dtype=dtype, device=DEV) for _ in range(2))
    got = rq.kv_read(dev_cache(cache), table.to(DEV), starts.to(DEV), offsets.to(DEV), total, SEED, flags, dtype=dtype, out=out)
    R = ref.rotation(D, SEED, flags & 1)
    for n, g in zip("kv", got):
        assert (g[int(offsets[-1]):] == 7.0).all()
        for b, cnt in enumerate(counts):
            for i in range(cnt):
                pos = int(starts[b]) + i
                pg = int(table[b, pos // page]) if pos // page < W else -1
                row = g[int(offsets[b]) + i].cpu().double()
                if pg < 0 or pg >= pages:
                    assert (row == 0).all()
                    continue
                want = ref.decode(cache[n + "q"][pg, :, pos % page], cache[n + "s"][pg, :, pos % page])
                if not flags & 2:
                    want = want @ R.T
                u = 0.0 if dtype == torch.float32 else ref.UNIT[dtype] * 1.02
                small = 2.0**-25 if dtype == torch.float16 else 0.0
                scale = cache[n + "s"][pg, :, pos % page].double()[:, None]
                # relative to the exact sum; where it cancels to 0 the fp64 reference itself carries 1e-15
                assert ((row - want).abs() <= (4e-7 + u) * want.abs() + small + 1e-12 * scale).all()


# ------------------------------------------------------------------ tree attention

def paged(lens, H, page, D, seed, scale=1.0, spare=2):
    """A filled cache and block tables for sequences of the given lengths, pages in random order."""
    need = [max(1, -(-n // page)) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=gen(seed)).to(torch.int32)
    table = torch.full((len(lens), max(need) if need else 1), -5, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return filled_cache(pages, H, page, D, seed + 1, scale), table


def check_tree(q, cache, table, contexts, counts, flags=1, mask=None, scale=None, max_nodes=None, **kw):
    D = q.shape[-1]
    contexts = torch.tensor(contexts, dtype=torch.int32)
    offsets = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)
    sc = D ** -0.5 if scale is None else scale
    got = rq.attn_tree(q.to(DEV), dev_cache(cache), table.to(DEV), contexts.to(DEV), offsets.to(DEV), SEED, flags,
                       tree_mask=None if mask is None else mask.to(DEV), softmax_scale=scale,
                       max_nodes=max_nodes if max_nodes is not None else (None if mask is not None else max(counts)), **kw)
    assert got.dtype == q.dtype and got.shape == q.shape
    want, spread, delta = ref.attention(q, cache, table, contexts, offsets, SEED, flags, sc, mask, rotated=bool(flags & 2))
    g = got.cpu().double()
    assert torch.isfinite(g).all()
    f32 = q.dtype == torch.float32
    part = 2.0**-22 if f32 else 2.0**-12
    eps = 8e-6 + 2 * part + 2 * (4 / 3) * part * delta
    u = ref.UNIT[q.dtype]
    err, bound = (g - want).norm(dim=-1), eps * spread.norm(dim=-1) + u * want.norm(dim=-1) + (2.0**-25 * D**0.5 if q.dtype == torch.float16 else 0)
    assert (err <= bound).all(), float((err / bound.clamp_min(1e-300)).max())
    return got


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,page", [(32, 16), (64, 32), (128, 64), (256, 128)])
@pytest.mark.parametrize("H,G,n", [(2, 1, 1), (1, 4, 5), (2, 8, 9), (1, 2, 33)])
def test_tree_shapes(dtype, D, page, H, G, n):
    counts, contexts = [n, max(1, n // 2), 1], [130, 77, 300]
    cache, table = paged([c + k for c, k in zip(contexts, counts)], H, page, D, 50 + n)
    q = randn(sum(counts), H * G, D, seed=51, dtype=dtype)
    check_tree(q, cache, table, contexts, counts, mask=ref.tree_mask(counts, gen(52)) if n > 1 else None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("context", [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 2000])
@pytest.mark.parametrize("n", [1, 7, 40])
def test_tree_lengths(dtype, context, n):
    """Contexts around the tiles' and pages' ends, from none; chains without a mask."""
    H, G, D = 2, 4, 128
    cache, table = paged([context + n], H, 16, D, 60 + context)
    check_tree(randn(n, H * G, D, seed=61, dtype=dtype), cache, table, [context], [n])


@pytest.mark.parametrize("flags", [0, 1, 2, 3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("n", [3, 48])
def test_tree_bases(flags, dtype, n):
    cache, table = paged([200 + n, 90 + n], 2, 32, 64, 70)
    check_tree(randn(2 * n, 8, 64, seed=71, dtype=dtype), cache, table, [200, 90], [n, n], flags=flags,
               mask=ref.tree_mask([n, n], gen(72)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("G,n", [(1, 4), (4, 40)])
def test_tree_empty_rows_and_sequences(dtype, G, n):
    """A sequence without nodes, one without context whose mask leaves rows empty (zeros), and poisoned places that
    no row may see: masked nodes, the rest of the last page, pages of nobody."""
    H, D, page = 2, 128, 32
    counts, contexts = [n, 0, n, 1], [100, 50, 0, 0]
    cache, table = paged([c + k for c, k in zip(contexts, counts)], H, page, D, 80)
    mask = ref.tree_mask(counts, gen(81))
    first = counts[0]
    mask[first:first + 2] = False                                # nothing visible: context 0
    mask[:, 2] = False                                           # node 2 is hidden from all
    mask[first + n] = False
    used = torch.zeros(cache["ks"].shape[0], page, dtype=torch.bool)
    for b, (c, k) in enumerate(zip(contexts, counts)):
        pg, row = ref.places(table, page, b, c + k)
        used[pg, row] = True
        if k > 2:
            used[pg[c + 2], row[c + 2]] = False
    for name in ("ks", "vs"):
        bad = torch.tensor([float("nan"), float("inf"), float("-inf"), 3e38])
        t = cache[name].transpose(1, 2)
        t[~used] = bad[torch.arange(int((~used).sum())) % 4][:, None].expand(-1, H)
    q = randn(sum(counts), H * G, D, seed=82, dtype=dtype)
    got = check_tree(q, cache, table, contexts, counts, mask=mask)
    assert (got[first:first + 2] == 0).all() and (got[first + n] == 0).all()


@pytest.mark.parametrize("n", [2, 40])
def test_tree_bad_pages_are_not_seen(n):
    """Page numbers outside the cache and contexts past the table drop out, like masked tokens."""
    H, D, page = 1, 64, 16
    cache, table = paged([200], H, page, D, 90)
    table[0, 3], table[0, 7] = -1, cache["ks"].shape[0]
    check_tree(randn(n, 4, D, seed=91, dtype=torch.bfloat16), cache, table, [150], [n])
    check_tree(randn(n, 4, D, seed=92, dtype=torch.bfloat16), cache, table, [5000], [n])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [3, 36])
@pytest.mark.parametrize("kind", ["sharp", "flat", "tiny_values", "huge_values", "uneven_values", "large_queries"])
def test_tree_magnitudes(dtype, n, kind):
    H, G, D = 1, 4, 128
    cache, table = paged([700 + n], H, 64, D, 100)
    scale, qs = None, 1.0
    if kind == "sharp":
        scale = 0.6
    if kind == "flat":
        scale = 0.0
    if kind == "tiny_values":
        cache["vs"] *= 1e-9 if dtype != torch.float16 else 1e-2
    if kind == "huge_values":
        cache["vs"] *= 1e9 if dtype != torch.float16 else 1e3
    if kind == "uneven_values":      # value rows over 2^20, the largest late
        cache["vs"] *= torch.exp2(-20.0 * torch.rand(cache["vs"].shape, generator=gen(101)))
    if kind == "large_queries":
        scale, qs = 1e-4, 3000.0
    check_tree(randn(n, H * G, D, seed=102, dtype=dtype, scale=qs), cache, table, [700], [n], scale=scale)


@pytest.mark.parametrize("n", [1, 6, 50])
def test_tree_strided_queries_streams_and_repeats(n):
    """q as a slice of a projection's rows, on another stream; two calls give the same bits; a caller's workspace."""
    H, G, D, page, B = 4, 2, 128, 64, 6
    contexts, counts = [500 + 37 * b for b in range(B)], [n] * B
    cache, table = paged([c + n for c in contexts], H, page, D, 110)
    rows = randn(B * n, (H * G + 2 * H) * D, seed=111, dtype=torch.bfloat16).to(DEV)
    q = rows[:, :H * G * D].view(B * n, H * G, D)
    mask = ref.tree_mask(counts, gen(112))
    want = check_tree(q.cpu(), cache, table, contexts, counts, mask=mask)
    dc, tb = dev_cache(cache), table.to(DEV)
    ctx = torch.tensor(contexts, dtype=torch.int32, device=DEV)
    off = torch.arange(0, B * n + 1, n, dtype=torch.int32, device=DEV)
    wide = torch.zeros(B * n, n + 5, dtype=torch.bool, device=DEV)
    wide[:, :n] = mask.to(DEV)
    ws = torch.empty(rq.attn_tree_workspace(D) + 16, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = rq.attn_tree(q, dc, tb, ctx, off, SEED, 1, tree_mask=wide[:, :n], stream=s, workspace=ws)
    again = rq.attn_tree(q, dc, tb, ctx, off, SEED, 1, tree_mask=wide, max_nodes=n, stream=s, workspace=ws)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(again, want)


@pytest.mark.parametrize("G", [1, 8])
def test_tree_matches_attn_decode(G):
    """One node and one query head per KV head: the dense cache's decode attention on the same rows."""
    H, D, page, T = 4, 128, 64, 640
    k, v = randn(T, H, D, seed=120, dtype=torch.bfloat16).to(DEV), randn(T, H, D, seed=121, dtype=torch.bfloat16).to(DEV)
    q = randn(1, H * G, D, seed=122).to(DEV)
    dense = rq.kv_rotate_quant(k, v, SEED, 1)
    cache = {n: t.view(T // page, page, H, -1).transpose(1, 2).reshape(T // page, H, page, -1).contiguous() for n, t in dense.items()}
    cache["ks"], cache["vs"] = cache["ks"][..., 0].contiguous(), cache["vs"][..., 0].contiguous()
    table = torch.arange(T // page, dtype=torch.int32, device=DEV)[None]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    got = rq.attn_tree(q, cache, table, i32(T - 1), i32(0, 1), SEED, 1)
    for g in range(G):
        want = rq.attn_decode(q[:, g::G].contiguous(), dense, SEED, 1)
        torch.testing.assert_close(got[:, g::G], want, rtol=1e-4, atol=1e-4 * float(want.abs().max()))


def test_many_sequences():
    """More sequences than the schedule scans one by one, some without nodes."""
    B, H, D, page = 300, 1, 64, 16
    g = gen(130)
    contexts = torch.randint(0, 60, (B,), generator=g).tolist()
    counts = torch.randint(0, 3, (B,), generator=g).tolist()
    cache, table = paged([c + n for c, n in zip(contexts, counts)], H, page, D, 131)
    check_tree(randn(sum(counts), 2, D, seed=132, dtype=torch.bfloat16), cache, table, contexts, counts, max_nodes=2)


def test_verification_step_end_to_end():
    """rope -> kv_append -> attn_tree -> kv_read, against the 64-bit attention on the rows that were read back."""
    H, G, D, page, ctx, n = 2, 4, 128, 32, 150, 9
    turns, m = rq.rope_turns(D, device=DEV)
    cache = rq.kv_cache(8, H, D, page)
    table = torch.tensor([[6, 2, 4, 0, 7, 5]], dtype=torch.int32, device=DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    pos = torch.arange(ctx + n, device=DEV)
    slots = table[0].long()[pos // page] * page + pos % page
    k, v = randn(ctx + n, H, D, seed=140, dtype=torch.bfloat16).to(DEV), randn(ctx + n, H, D, seed=141, dtype=torch.bfloat16).to(DEV)
    rq.kv_append(k[:ctx], v[:ctx], cache, slots[:ctx], SEED, 1, positions=pos[:ctx], turns=turns)
    mask = ref.tree_mask([n], gen(142))
    depth = mask.sum(1).to(DEV) - 1
    rq.kv_append(k[ctx:], v[ctx:], cache, slots[ctx:], SEED, 1, positions=ctx + depth, turns=turns)
    q, _ = rq.rope(randn(n, H * G, D, seed=143, dtype=torch.bfloat16).to(DEV), None, ctx + depth, turns)
    out = rq.attn_tree(q, cache, table, i32(ctx), i32(0, n), SEED, 1, tree_mask=mask.to(DEV))
    kd, vd = rq.kv_read(cache, table, None, i32(0, ctx + n), ctx + n, SEED, 1, dtype=torch.float32)
    seen = torch.cat([torch.ones(n, ctx, dtype=torch.bool), mask], 1).to(DEV)
    for h in range(H * G):
        s = (q[:, h].double() @ kd[:, h // G].double().T) * D ** -0.5
        want = torch.softmax(s.masked_fill(~seen, -np.inf), -1) @ vd[:, h // G].double()
        err = (out[:, h].double() - want).norm(dim=-1) / want.norm(dim=-1)
        assert err.max() < 6e-3           # bf16 rounding up to 2^-8 of each element, weights 2^-11


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,H,G,n,context,D,page", [
    (64, 8, 2, 10, 200, 128, 16),      # whole blocks of rows and pieces of them in one thread block
    (16, 8, 2, 12, 1300, 64, 32),      # stretches of many tiles
    (5, 4, 8, 40, 1500, 128, 64),      # more than 256 rows
    (24, 2, 4, 33, 700, 128, 256),     # a little more than 128 rows
    (40, 8, 1, 3, 900, 64, 64),        # few rows
    (9, 4, 4, 1, 5000, 128, 128),      # single tokens
])
def test_tree_many_tiles(dtype, B, H, G, n, context, D, page):
    """More tiles than thread blocks: stretches that begin and end inside sequences, heads and row blocks."""
    g = gen(150 + B)
    contexts = (torch.rand(B, generator=g) * context).to(torch.int32).tolist()
    counts = torch.randint(max(1, n - 3), n + 1, (B,), generator=g).tolist()
    counts[0] = n
    cache, table = paged([c + k for c, k in zip(contexts, counts)], H, page, D, 151)
    cache, table = dev_cache(cache), table.to(DEV)
    mask = ref.tree_mask(counts, g).to(DEV)
    q = randn(sum(counts), H * G, D, seed=152, dtype=dtype).to(DEV)
    offsets = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)
    ctx = torch.tensor(contexts, dtype=torch.int32, device=DEV)
    want, spread, delta = ref.attention_blocks(q, cache, table, contexts, offsets, SEED, 1, D ** -0.5, mask)
    got = rq.attn_tree(q, cache, table, ctx, offsets, SEED, 1, tree_mask=mask)
    part = 2.0**-22 if dtype == torch.float32 else 2.0**-12
    eps = 8e-6 + 2 * part + 2 * (4 / 3) * part * delta
    bound = eps * spread.norm(dim=-1) + ref.UNIT[dtype] * want.norm(dim=-1) + (2.0**-25 * D**0.5 if dtype == torch.float16 else 0)
    err = (got.double() - want).norm(dim=-1)
    assert (err <= bound).all(), float((err / bound).max())
    assert torch.equal(got, rq.attn_tree(q, cache, table, ctx, offsets, SEED, 1, tree_mask=mask))
