"""A decode step of requests that share a prompt, as workloads to time and to compare.

Three operators: block tables and slots made on the GPU from the requests' lengths (``plan``),
attention over the paged INT4 cache where groups of sequences share a prefix that is read once
for all of them (``prefix``), and products of a few 16- or 32-bit rows with 4-bit weights and
group scales (``matvec``).  ``run`` takes one pass through one of them: in the plain form
(elementary torch operations in 32 bits, rounded once at the end), or, where ``own`` is true,
through the framework's entry points.
"""
import math

import numpy as np
import torch

own = False

SEED = 0x5EED          # sign vector of the head-wise rotation
FLAGS = 1              # signs act first
GROUP = 128            # weights that share a scale
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
DEV = "cuda"


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # every step of a decode loop: one new token for each of 64 running requests
        dict(name="plan_decode", op="plan", seqs=64, new=1, context=8192, page=64, pad=0, shared=1024, short=False),
        # a large batch of prompts enters, ragged and padded to a fixed number of rows; small pages
        dict(name="plan_prompts", op="plan", seqs=509, new=768, context=512, page=16, pad=4099, shared=0, short=False),
        # the smallest call: one token's key projection
        dict(name="matvec_small", op="matvec", rows=1, k=4096, n=1024, dtype="bf16", out="bf16", grouped=True),
        # one token through an up projection
        dict(name="matvec_up", op="matvec", rows=1, k=4096, n=14336, dtype="bf16", out="bf16", grouped=True),
        # a few drafted tokens through a down projection, fp16
        dict(name="matvec_down", op="matvec", rows=7, k=14336, n=4096, dtype="f16", out="f16", grouped=True),
        # fp32 rows as the rotation leaves them, one scale per channel, an odd number of channels
        dict(name="matvec_f32", op="matvec", rows=3, k=4096, n=4101, dtype="f32", out="f32", grouped=False),
        # a batch of 61 requests, one token each, through the up projection
        dict(name="matvec_batch", op="matvec", rows=61, k=4096, n=14336, dtype="bf16", out="bf16", grouped=True),
        # a decode batch through the largest layer
        dict(name="matvec_large", op="matvec", rows=16, k=8192, n=28672, dtype="bf16", out="f16", grouped=True),
        # four samples of one short prompt, a few tokens in: the smallest attention
        dict(name="prefix_small", op="prefix", seqs=4, groups=1, prefix=1000, own=37, nodes=1, heads=32, kv_heads=8,
             dim=128, page=16, dtype="f16", mask=False),
        # a serving batch with a common system prompt, one token each
        dict(name="prefix_decode", op="prefix", seqs=64, groups=1, prefix=8192, own=512, nodes=1, heads=32, kv_heads=8,
             dim=128, page=64, dtype="bf16", mask=False),
        # several prompts of uneven length (one group has none), drafted trees on top, multi-head fp32 with small heads
        dict(name="prefix_trees", op="prefix", seqs=21, groups=5, prefix=3001, own=130, nodes=5, heads=16, kv_heads=16,
             dim=64, page=32, dtype="f32", mask=True),
        # many requests over one long document: the largest call
        dict(name="prefix_long", op="prefix", seqs=256, groups=2, prefix=32768, own=2048, nodes=1, heads=64, kv_heads=8,
             dim=128, page=64, dtype="bf16", mask=False),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "matvec", "matvec", "prefix", "prefix"])
    if op == "plan":
        seqs = _log_uniform(rng, 1, 1024)
        new = _log_uniform(rng, 1, max(1, min(8192, 390000 // seqs)))
        return dict(op="plan", seqs=seqs, new=new, context=_log_uniform(rng, 1, 16384), page=rng.choice([16, 32, 64, 128]),
                    pad=rng.choice([0, 0, _log_uniform(rng, 1, 4096)]), shared=rng.choice([0, _log_uniform(rng, 1, 8192)]),
                    short=rng.random() < 0.15)
    if op == "matvec":
        k = 128 * _log_uniform(rng, 1, 224)
        n = _log_uniform(rng, 1, min(28672, 8192 * 28672 // k))
        return dict(op="matvec", rows=rng.choice([1, _log_uniform(rng, 1, 64)]), k=k, n=n,
                    dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), out=rng.choice(["bf16", "f16", "f32"]),
                    grouped=rng.random() < 0.75)
    kv = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 2, 4, 4, 8])
    dim = rng.choice([32, 64, 128, 128, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
    seqs = _log_uniform(rng, 1, 256)
    nodes = rng.choice([1, 1, 1, _log_uniform(rng, 1, 16)])
    slow = 4 if dtype == "f32" or dim in (32, 256) else 1
    most = 256 * 34816 * 64 * 128 // (seqs * nodes * kv * group * dim * slow)               # tokens seen, by products
    own_most = min(most // 2, 256 * 2048 * 8 * 128 // (seqs * kv * dim))                    # and by bytes
    return dict(op="prefix", seqs=seqs, groups=_log_uniform(rng, 1, min(seqs, 8)),
                prefix=_log_uniform(rng, 1, max(1, min(65536, most - own_most))), own=_log_uniform(rng, 1, max(1, min(4096, own_most))),
                nodes=nodes, heads=kv * group, kv_heads=kv, dim=dim, page=rng.choice([16, 32, 64, 128]), dtype=dtype,
                mask=nodes > 1 and rng.random() < 0.7)


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _signs(n):
    """+-1 by the top bit of the first n outputs of SplitMix64(SEED)."""
    out, mask = [], (1 << 64) - 1
    for i in range(n):
        z = (SEED + (i + 1) * 0x9E3779B97F4A7C15) & mask
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & mask
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
        out.append(-1.0 if (z ^ (z >> 31)) >> 63 else 1.0)
    return out


def _rotation(n):
    """R = diag(s) H / sqrt(n) in fp64, on the CPU."""
    h = np.array([[1.0]])
    while h.shape[0] < n:
        h = np.block([[h, h], [h, -h]])
    return np.array(_signs(n))[:, None] * h / math.sqrt(n)


def _spread(n, most, least):
    """n ragged sizes from `least` times `most` up to `most`, which the first has: the same ones for every seed."""
    r = np.random.RandomState(n + most).rand(n)
    return [most] + [int(most * (least + (1 - least) * x)) for x in r[1:]]


def _codes_of(y):
    """Rows of y (last dimension) as packed 4-bit codes and fp32 scales, max / 7."""
    top = y.abs().amax(-1)
    q = (y * (7.0 / top)[..., None]).round_().to(torch.int8)
    return ((q[..., 0::2] & 15) | (q[..., 1::2] << 4)).view(torch.uint8), top / 7.0


def _filled_cache(g, pages, heads, page, dim):
    """A cache that holds quantised normal rows of uneven magnitude."""
    cache = {}
    for name in ("k", "v"):
        codes = torch.empty(pages, heads, page, dim // 2, dtype=torch.uint8, device=DEV)
        scales = torch.empty(pages, heads, page, dtype=torch.float32, device=DEV)
        step = max(1, (1 << 27) // (heads * page * dim))
        for a in range(0, pages, step):
            b = min(pages, a + step)
            y = torch.randn(b - a, heads, page, dim, generator=g, device=DEV)
            codes[a:b], top = _codes_of(y)
            scales[a:b] = top * torch.exp(0.3 * torch.randn(top.shape, generator=g, device=DEV))
        cache[name + "q"], cache[name + "s"] = codes, scales
    return cache


def _plan_lengths(case):
    """Tokens that each request has in the cache, and new ones: a few requests are fresh, a few have nothing to do."""
    contexts, new = _spread(case["seqs"], case["context"], 0.0), _spread(case["seqs"], case["new"], 0.2)
    contexts = [0 if b % 7 == 3 else c for b, c in enumerate(contexts)]
    new = [0 if b % 11 == 5 else max(1, n) for b, n in enumerate(new)]
    return contexts, new


def _pages(n, page):
    return -(-n // page)


def _prefix_shape(case):
    """Sequences of each group, its prefix (the last of several has none), tokens of each sequence before its nodes."""
    sizes = _spread(case["groups"], max(1, case["seqs"] // case["groups"]), 0.5)
    sizes = [max(1, s) for s in sizes]
    sizes[0] += case["seqs"] - sum(sizes)
    prefixes = _spread(case["groups"], case["prefix"], 0.3)
    if case["groups"] > 2:
        prefixes[-1] = 0
    own_tokens = [max(0, n - case["nodes"]) for n in _spread(case["seqs"], case["own"], 0.0)]
    return sizes, prefixes, own_tokens


def _table(order, lengths, page):
    """Block tables that take their pages from `order`, and what is left of it."""
    need = [_pages(n, page) for n in lengths]
    table, at = torch.zeros(len(lengths), max(1, max(need)), dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table.to(DEV), order[at:]


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    if case["op"] == "plan":
        contexts, new = _plan_lengths(case)
        page, total = case["page"], sum(new) + case["pad"]
        kept = [_pages(c, page) for c in contexts]
        wanted = sum(_pages(c + n, page) for c, n in zip(contexts, new)) - sum(kept)
        width = max(_pages(c + n, page) for c, n in zip(contexts, new)) + 1
        order = torch.randperm(sum(kept) + 2 * wanted + 8, generator=g, device=DEV).to(torch.int32).cpu()
        table, at = torch.full((case["seqs"], width), -1, dtype=torch.int32), 0
        for b, n in enumerate(kept):
            table[b, :n] = order[at:at + n]
            at += n
        # pages that earlier steps took lie before the head of the free list
        taken = wanted // 3
        free = order[at:at + taken + (wanted * 3 // 4 + 1 if case["short"] else wanted + 5)]
        s.update(contexts=_i32(contexts), new=_i32(new), table=table.to(DEV), free=free.to(DEV), head=_i32([taken]), total=total)
        s["base"] = torch.full((case["seqs"],), case["shared"], dtype=torch.int32, device=DEV) if case["shared"] else None
        return s
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "matvec":
        n, k = case["n"], case["k"]
        group = GROUP if case["grouped"] else k
        codes = torch.empty(n, k // 2, dtype=torch.uint8, device=DEV)
        scales = torch.empty(n, k // group, dtype=torch.float32, device=DEV)
        step = max(1, (1 << 27) // k)
        for a in range(0, n, step):
            w = 0.02 * torch.randn(min(n, a + step) - a, k // group, group, generator=g, device=DEV)
            q, scales[a:a + step] = _codes_of(w)
            codes[a:a + step] = q.flatten(1)
        # rotated activations: near normal, rows of uneven magnitude
        x = torch.randn(case["rows"], k, generator=g, device=DEV)
        x *= torch.exp(torch.randn(case["rows"], 1, generator=g, device=DEV))
        s.update(x=x.to(dtype), w=codes, scales=scales if case["grouped"] else scales[:, 0].contiguous())
        return s
    page, nodes = case["page"], case["nodes"]
    sizes, prefixes, own_tokens = _prefix_shape(case)
    lengths = [n + nodes for n in own_tokens]
    count = sum(_pages(n, page) for n in lengths) + sum(_pages(n, page) for n in prefixes)
    order = torch.randperm(count, generator=g, device=DEV).to(torch.int32).cpu()
    s["prefix_table"], order = _table(order, prefixes, page)
    s["table"], _ = _table(order, lengths, page)
    s["cache"] = _filled_cache(g, count, case["kv_heads"], page, case["dim"])
    rows = case["seqs"] * nodes
    s["q"] = (1.5 * torch.randn(rows, case["heads"], case["dim"], generator=g, device=DEV)).to(dtype)
    s["contexts"], s["offsets"] = _i32(own_tokens), _i32(list(range(0, rows + 1, nodes)))
    s["prefix_lens"], s["groups"] = _i32(prefixes), _i32([0] + list(np.cumsum(sizes)))
    s["mask"] = None
    if case["mask"]:
        mask, r = np.zeros((rows, nodes), dtype=bool), torch.rand(rows, generator=g, device=DEV).cpu().numpy()
        for at in range(0, rows, nodes):
            for i in range(nodes):
                if i:      # a parent among the nodes before it
                    mask[at + i] = mask[at + int(r[at + i] * i)]
                mask[at + i, i] = True
        s["mask"] = torch.tensor(mask, device=DEV)
    s["rotation"] = torch.tensor(_rotation(case["dim"]), dtype=torch.float32, device=DEV)
    # what the plain form's loop over groups goes by
    s["spans"], at = [], 0
    for size, n in zip(sizes, prefixes):
        s["spans"].append((at * nodes, (at + size) * nodes, n))
        at += size
    s["longest"] = max(lengths)
    return s


# ---------------------------------------------------------------- the plain forms, in 32 bits

def _plain_plan(s):
    page, table, free = s["case"]["page"], s["table"], s["free"]
    seqs, width = table.shape
    contexts, ends = s["contexts"].long(), (s["contexts"] + s["new"]).long()
    kept, need = (contexts + page - 1) // page, (ends + page - 1) // page
    first = torch.cumsum(need - kept, 0) - (need - kept) + s["head"].long()            # of each request, in the free list
    column = torch.arange(width, device=DEV)[None, :]
    at = first[:, None] + column - kept[:, None]
    fresh = torch.where(at < free.numel(), free[at.clamp(0, free.numel() - 1)], -1)
    table.copy_(torch.where(column < kept[:, None], table, torch.where(column < need[:, None], fresh, -1)))
    offsets = torch.zeros(seqs + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.cumsum(s["new"].long(), 0)
    row = torch.arange(s["total"], device=DEV)
    seq = (torch.searchsorted(offsets, row, right=True) - 1).clamp(max=seqs - 1)
    there = row < offsets[-1]
    place = torch.where(there, row - offsets[seq] + contexts[seq], 0)
    number = table[seq, (place // page).clamp(max=width - 1)].long()
    slots = torch.where(there & (number >= 0), number * page + place % page, -1)
    positions = place if s["base"] is None else torch.where(there, place + s["base"][seq], 0)
    head = (s["head"].long() + (need - kept).sum()).to(torch.int32)
    return {"offsets": offsets.to(torch.int32), "slots": slots, "positions": positions, "head": head, "table": table}


def _plain_codes(b):
    q = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    return ((q ^ 8).to(torch.int8) - 8).float()


def _plain_matvec(s):
    case = s["case"]
    w = _plain_codes(s["w"]).view(case["n"], -1, GROUP if case["grouped"] else case["k"])
    w *= s["scales"].view(case["n"], -1, 1)
    return (s["x"].float() @ w.flatten(1).T).to(DTYPES[case["out"]])


def _plain_rows(cache, name, pages, rows):
    """Cache rows (page, row of the page) as values in the rotated basis: [..., heads, dim]."""
    return _plain_codes(cache[name + "q"][pages, :, rows]) * cache[name + "s"][pages, :, rows][..., None]


def _plain_prefix(s):
    case, cache, nodes = s["case"], s["cache"], s["case"]["nodes"]
    seqs, heads, kv, d, page = (case[k] for k in ("seqs", "heads", "kv_heads", "dim", "page"))
    group, rows = heads // kv, seqs * nodes
    q = (s["q"].float() @ s["rotation"]).view(rows, kv, group, d) * d ** -0.5
    # each sequence's own tokens, padded to the longest
    at = torch.arange(s["longest"], device=DEV)
    pages, row = s["table"][:, at // page].long(), (at % page).expand(seqs, -1)
    k = _plain_rows(cache, "k", pages, row).permute(0, 2, 3, 1)                    # [seqs, kv, d, longest]
    scores = q.view(seqs, nodes, kv, group, d).permute(0, 2, 1, 3, 4).reshape(seqs, kv, nodes * group, d) @ k
    node = at[None, :] - s["contexts"][:, None]                                    # the node at each place
    if s["mask"] is None:
        seen = node[:, None, :] <= torch.arange(nodes, device=DEV)[None, :, None]
    else:
        mask = s["mask"].view(seqs, nodes, nodes)
        seen = torch.gather(mask, 2, node.clamp(0, nodes - 1)[:, None, :].expand(-1, nodes, -1))
        seen = (node < 0)[:, None, :] | (seen & (node < nodes)[:, None, :])
    seen = seen[:, None, :, None, :].expand(-1, kv, -1, group, -1).reshape(seqs, kv, nodes * group, -1)
    scores = torch.where(seen, scores, -torch.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -torch.inf, 0.0, top))
    o = p @ _plain_rows(cache, "v", pages, row).permute(0, 2, 1, 3)

    def by_row(x):                                                                 # -> [kv, rows, group, ...]
        return x.view(seqs, kv, nodes, group, -1).permute(1, 0, 2, 3, 4).reshape(kv, rows, group, -1)

    o, top, total = by_row(o), by_row(top), by_row(p.sum(-1, keepdim=True))
    q = q.permute(1, 0, 2, 3)
    # the prefixes, each for all rows of its group at once
    for i, (a, b, n) in enumerate(s["spans"]):
        if n == 0:
            continue
        at = torch.arange(n, device=DEV)
        pages, row = s["prefix_table"][i, at // page].long(), at % page
        scores = q[:, a:b].reshape(kv, -1, d) @ _plain_rows(cache, "k", pages, row).permute(1, 2, 0)
        top_here = scores.amax(-1, keepdim=True)
        p = torch.exp(scores - top_here)
        o_here = (p @ _plain_rows(cache, "v", pages, row).transpose(0, 1)).view(kv, b - a, group, d)
        total_here, top_here = p.sum(-1).view(kv, b - a, group, 1), top_here.view(kv, b - a, group, 1)
        both = torch.maximum(top[:, a:b], top_here)
        f, f_here = torch.exp(top[:, a:b] - both), torch.exp(top_here - both)
        o[:, a:b] = o[:, a:b] * f + o_here * f_here
        total[:, a:b] = total[:, a:b] * f + total_here * f_here
    return ((o / total) @ s["rotation"].T).permute(1, 0, 2, 3).reshape(rows, heads, d).to(DTYPES[case["dtype"]])


def run(s):
    case = s["case"]
    if own:
        import rotational_w4a4_quantization_gb300 as rq
        if case["op"] == "plan":
            offsets, slots, positions, head = rq.kv_plan(s["contexts"], s["new"], s["table"], s["free"], s["total"],
                                                         case["page"], head=s["head"], base=s["base"])
            return {"offsets": offsets, "slots": slots, "positions": positions, "head": head, "table": s["table"]}
        if case["op"] == "matvec":
            return rq.w4a16_gemm(s["x"], s["w"], s["scales"], out_dtype=DTYPES[case["out"]])
        return rq.attn_prefix(s["q"], s["cache"], s["table"], s["contexts"], s["offsets"], s["prefix_table"],
                              s["prefix_lens"], s["groups"], SEED, FLAGS, tree_mask=s["mask"], max_nodes=case["nodes"])
    if case["op"] == "plan":
        return _plain_plan(s)
    if case["op"] == "matvec":
        return _plain_matvec(s)
    return _plain_prefix(s)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "plan":
        contexts, new = _plan_lengths(case)
        page, total = case["page"], sum(new) + case["pad"]
        width = max(_pages(c + n, page) for c, n in zip(contexts, new)) + 1
        kept, need = sum(_pages(c, page) for c in contexts), sum(_pages(c + n, page) for c, n in zip(contexts, new))
        written = case["seqs"] * width - kept                                      # table entries: those behind the kept
        # kept entries are read where a request's first new token falls into them
        read = sum(1 for c, n in zip(contexts, new) if n and c % page) + need - kept
        return {"bytes": 16 * total + 4 * (written + read + 4 * case["seqs"]), "flops": 4 * total}
    size = BYTES[case["dtype"]]
    if case["op"] == "matvec":
        m, n, k = case["rows"], case["n"], case["k"]
        scales = n * (k // GROUP if case["grouped"] else 1)
        return {"bytes": n * k // 2 + 4 * scales + m * k * size + m * n * BYTES[case["out"]], "flops": 2 * m * n * k}
    sizes, prefixes, own_tokens = _prefix_shape(case)
    d, kv, heads, nodes = case["dim"], case["kv_heads"], case["heads"], case["nodes"]
    tokens = sum(prefixes) + sum(own_tokens) + nodes * case["seqs"]
    seen = nodes * (sum(n * p for n, p in zip(sizes, prefixes)) + sum(own_tokens) + nodes * case["seqs"])
    return {"bytes": tokens * kv * (d + 8) + 2 * case["seqs"] * nodes * heads * d * size, "flops": 4 * seen * heads * d}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_plan(s):
    """Request by request, token by token."""
    page, contexts, new = s["case"]["page"], s["contexts"].tolist(), s["new"].tolist()
    table, free, at = s["table"].cpu().numpy().copy(), s["free"].tolist(), int(s["head"])
    base = [0] * len(new) if s["base"] is None else s["base"].tolist()
    slots, positions = np.full(s["total"], -1, dtype=np.int64), np.zeros(s["total"], dtype=np.int64)
    offsets = [0]
    for b, (c, n) in enumerate(zip(contexts, new)):
        have, want = _pages(c, page), _pages(c + n, page)
        for j in range(have, want):
            table[b, j] = free[at] if at < len(free) else -1
            at += 1
        table[b, want:] = -1
        for t in range(c, c + n):
            number = int(table[b, t // page])
            slots[offsets[-1] + t - c] = number * page + t % page if number >= 0 else -1
            positions[offsets[-1] + t - c] = t + base[b]
        offsets.append(offsets[-1] + n)
    return {"offsets": _i32(offsets), "slots": torch.from_numpy(slots).to(DEV), "positions": torch.from_numpy(positions).to(DEV),
            "head": _i32([at]), "table": torch.from_numpy(table).to(DEV)}


def _exact_values(codes, scales):
    """scales: one for each last dimension of the codes."""
    low = (codes & 15).double()
    high = torch.div(codes, 16, rounding_mode="floor").double()
    q = torch.stack([low, high], -1).flatten(-2)
    return torch.where(q > 7.5, q - 16.0, q) * scales.double()[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(s)
    if case["op"] == "matvec":
        n, x, out = case["n"], s["x"].double(), []
        step = max(1, (1 << 26) // case["k"])
        for a in range(0, n, step):
            scales = s["scales"][a:a + step].reshape(min(step, n - a), -1)
            codes = s["w"][a:a + step].reshape(scales.shape[0], scales.shape[1], -1)
            out.append(torch.einsum("mk,nk->mn", x, _exact_values(codes, scales).flatten(1)))
        return torch.cat(out, 1)
    r = torch.tensor(_rotation(case["dim"]), device=DEV)
    page, nodes, cache = case["page"], case["nodes"], s["cache"]
    contexts, prefixes, groups = s["contexts"].tolist(), s["prefix_lens"].tolist(), s["groups"].tolist()
    heads_each = case["heads"] // case["kv_heads"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)

    def values(name, table, h, count):
        used = table[:_pages(count, page)].long()
        return _exact_values(cache[name + "q"][used, h].flatten(0, 1), cache[name + "s"][used, h].flatten())[:count] @ r.T

    for i, n in enumerate(prefixes):
        for h in range(case["kv_heads"]):
            kp, vp = (values(name, s["prefix_table"][i], h, n) for name in ("k", "v"))
            for b in range(groups[i], groups[i + 1]):
                rows, count = slice(b * nodes, (b + 1) * nodes), contexts[b] + nodes
                seen = torch.ones(nodes, n + count, dtype=torch.bool, device=DEV)
                seen[:, n + contexts[b]:] = torch.ones_like(seen[:, :nodes]).tril() if s["mask"] is None else s["mask"][rows]
                ks, vs = (values(name, s["table"][b], h, count) for name in ("k", "v"))
                q = s["q"][rows, h * heads_each:(h + 1) * heads_each].double()
                score = torch.cat([torch.einsum("ngd,td->ngt", q, kp), torch.einsum("ngd,td->ngt", q, ks)], -1)
                p = torch.softmax((score / math.sqrt(case["dim"])).masked_fill(~seen[:, None, :], -math.inf), -1)
                out[rows, h * heads_each:(h + 1) * heads_each] = (torch.einsum("ngt,td->ngd", p[..., :n], vp)
                                                                  + torch.einsum("ngt,td->ngd", p[..., n:], vs))
    return out
