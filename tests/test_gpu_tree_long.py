"""Tree attention where one thread block sums very many tokens: more (sequence, KV head) pairs than blocks, long contexts
on shared pages."""
import pytest
import torch

import paged_ref as ref
import rotational_w4a4_quantization_gb300 as rq
from test_gpu_paged import DEV, SEED, _built, _status, gen  # noqa: F401

pytestmark = pytest.mark.gpu
D, PAGE = 64, 128
# sequences, query heads (one KV head), nodes: blocks of 8 and 16 rows, of 128, and (bf16) of 256
SHAPES = [(520, 1, 1), (520, 4, 3), (160, 4, 12), (160, 4, 40)]


def pack(codes):
    c = codes.to(torch.int64) & 15
    return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8)


def shared(N, seed, common=0):
    g = gen(seed)
    pages = -(-N // PAGE)
    shape = (pages, 1, PAGE)
    return {"kq": pack(torch.randint(-7, 8, (*shape, D), generator=g)).to(DEV),
            "ks": (0.03 + 0.04 * torch.rand(shape, generator=g)).to(DEV),
            "vq": pack(common + torch.randint(-3, 4, (*shape, D), generator=g)).to(DEV),
            "vs": (0.2 + 0.2 * torch.rand(shape, generator=g)).to(DEV)}, torch.arange(pages, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("B,G,n", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_lengths_around_the_pieces(B, G, n, dtype):
    """Contexts of 250 to 600 tiles, each sequence with its own; some rows against 64 bits."""
    if dtype == torch.float32 and n > 12:
        B = 40                                               # blocks of 16 rows only: ten to a sequence
    cache, pages = shared(600 * 128, 700)
    g = gen(701)
    contexts = torch.randint(250 * 128, 600 * 128 - n, (B,), generator=g)
    special = torch.tensor([0, 1, 256, 257, 512, 513, 256, 512]) * 128 + torch.tensor([0, 0, 0, 1, -n, 0, -n, 1])
    contexts[:8] = special.clamp(0, 600 * 128 - n)
    table = pages[None].repeat(B, 1)
    q = (torch.randn(B * n, G, D, generator=g) * 2).to(dtype).to(DEV)
    off = torch.arange(B + 1, dtype=torch.int32, device=DEV) * n
    got = rq.attn_tree(q, cache, table, contexts.to(torch.int32).to(DEV), off, SEED, max_nodes=n)
    part = 2.0**-22 if dtype == torch.float32 else 2.0**-12
    for b in [*range(8), B // 2, B - 1]:
        own = slice(b * n, (b + 1) * n)
        want, spread, delta = ref.attention_blocks(q[own], cache, table[b:b + 1].cpu(), [int(contexts[b])], [0, n], SEED, 1, D ** -0.5)
        eps = 8e-6 + (2 if dtype == torch.bfloat16 and n > 3 else 1) * (2 * part + 2 * (4 / 3) * part * delta)
        bound = eps * spread.norm(dim=-1) + ref.UNIT[dtype] * want.norm(dim=-1) + (2.0**-25 * D**0.5 if dtype == torch.float16 else 0)
        err = (got[own].double() - want).norm(dim=-1)
        assert (err <= bound).all(), (b, int(contexts[b]), float((err / bound).max()))
    assert torch.equal(got, rq.attn_tree(q, cache, table, contexts.to(torch.int32).to(DEV), off, SEED, max_nodes=n))


@pytest.mark.parametrize("B,G,n,dtype", [(*s, d) for s in SHAPES for d in (torch.bfloat16, torch.float16)]
                         + [(*s, torch.float32) for s in SHAPES[:2]])
def test_sums_of_a_common_sign(B, G, n, dtype):
    """262,144 tokens whose values have a common part, in the rotated basis: the mean error of the elements.  The tensor
    cores add 256 tiles at most into one sum, 8 times a tile (few rows: twice), and lose less than 2^-24 of it each time,
    of a sum that grows from nothing: 256 * 8 * 2^-24 / 2 = 6.1e-5 in the mean; the other roundings are to nearest, and
    their mean over hundreds of elements is far below their 1.3e-3 (bf16)."""
    N = 262144 - n
    cache, pages = shared(262144, 710, common=3)
    g = gen(711)
    q = torch.randn(n, G, D, generator=g).to(dtype).to(DEV)
    table = pages[None].expand(B, -1).contiguous()
    off = torch.arange(B + 1, dtype=torch.int32, device=DEV) * n
    ctx = torch.full((B,), N, dtype=torch.int32, device=DEV)
    out = rq.attn_tree(q.repeat(B, 1, 1), cache, table, ctx, off, SEED, 3, max_nodes=n)
    R = ref.rotation(D, SEED, 1).to(DEV)
    t = torch.arange(N + n, device=DEV)
    k, v = (ref.decode(cache[x + "q"][t // PAGE, 0, t % PAGE], cache[x + "s"][t // PAGE, 0, t % PAGE]) for x in "kv")
    want = torch.empty(n, G, D, dtype=torch.float64, device=DEV)
    for i in range(n):
        s = (q[i].double() @ R) @ k[:N + i + 1].T * D ** -0.5
        want[i] = torch.softmax(s, -1) @ v[:N + i + 1]
    for b in (0, B // 2, B - 1):
        mean = float(((out[b * n:(b + 1) * n].double() - want) / want).mean())
        noise = 4 * ref.UNIT[dtype] / (3 * n * G * D) ** 0.5          # four sigma of the outputs' own rounding
        assert abs(mean) < 6.1e-5 + noise, mean
