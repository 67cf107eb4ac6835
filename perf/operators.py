"""The serving operators of the rotated INT4 cache, as workloads to time and to compare.

Three operators: rotary positions on queries and keys (``rope``), a paged INT4 cache
that is quantised as it is written and read back dense (``cache``), and attention of
trees of drafted tokens over that cache (``tree``).  ``run`` takes one pass through one
of them: in the plain form (elementary torch operations in 32 bits, rounded once at the
end), or, where ``own`` is true, through the framework's entry points.
"""
import math

import numpy as np
import torch

own = False

SEED = 0x5EED          # sign vector of the head-wise rotation
FLAGS = 1              # signs act first
BASE = 10000.0
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
DEV = "cuda"


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # the rotary step of a decode batch: one new token for each of 16 sequences
        dict(name="rope_decode", op="rope", tokens=16, heads=32, kv_heads=8, dim=128, rot=128, layout="half",
             scaling="none", span=8192, dtype="bf16", inverse=False, fused_qkv=False),
        # the gradient of a rotary step: adjacent pairs, part of the head, fp32, an odd number of tokens
        dict(name="rope_grad_f32", op="rope", tokens=4099, heads=32, kv_heads=32, dim=64, rot=48, layout="interleaved",
             scaling="linear", span=16384, dtype="f32", inverse=True, fused_qkv=False),
        # a long prefill: q and k are slices of one projection's rows, frequencies scaled for a 16 times longer context
        dict(name="rope_long", op="rope", tokens=65536, heads=32, kv_heads=8, dim=128, rot=128, layout="half",
             scaling="parts", span=131072, dtype="bf16", inverse=False, fused_qkv=True),
        # a decode batch writes one token for each of 16 sequences and takes those back dense
        dict(name="cache_step", op="cache", seqs=16, new=1, context=1000, read_all=False, kv_heads=8, dim=128, page=64,
             dtype="bf16", rot=128, layout="half"),
        # chunked prefill: 2048 more tokens of an 8192-token sequence are written, the whole of it is read for a 16-bit attention
        dict(name="cache_chunk", op="cache", seqs=1, new=2048, context=6144, read_all=True, kv_heads=32, dim=128, page=64,
             dtype="bf16", rot=128, layout="half"),
        # many short ragged prompts, small pages that end inside every tile, half of the head rotary
        dict(name="cache_ragged", op="cache", seqs=48, new=333, context=517, read_all=True, kv_heads=8, dim=64, page=16,
             dtype="f16", rot=32, layout="interleaved"),
        # the smallest call: five drafted tokens of one short sequence
        dict(name="tree_small", op="tree", seqs=1, nodes=5, context=509, heads=32, kv_heads=8, dim=128, page=64,
             dtype="bf16", ragged=False, mask=True),
        # a plain decode step of 64 sequences, ragged contexts, eight query heads to a cache head
        dict(name="tree_decode", op="tree", seqs=64, nodes=1, context=8192, heads=64, kv_heads=8, dim=128, page=64,
             dtype="bf16", ragged=True, mask=False),
        # one token of two very long sequences: few rows, a long axis
        dict(name="tree_long", op="tree", seqs=2, nodes=1, context=262144, heads=32, kv_heads=8, dim=128, page=128,
             dtype="bf16", ragged=False, mask=False),
        # speculative verification of an ordinary batch: 16 nodes a sequence
        dict(name="tree_batch", op="tree", seqs=16, nodes=16, context=4096, heads=32, kv_heads=8, dim=128, page=32,
             dtype="f16", ragged=True, mask=True),
        # wide trees over long contexts: the largest call
        dict(name="tree_wide", op="tree", seqs=16, nodes=64, context=32768, heads=32, kv_heads=8, dim=128, page=64,
             dtype="bf16", ragged=True, mask=True),
        # multi-head fp32 with an odd tree and small heads
        dict(name="tree_f32", op="tree", seqs=5, nodes=13, context=2047, heads=16, kv_heads=16, dim=64, page=16,
             dtype="f32", ragged=True, mask=True),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "cache", "tree", "tree"])
    if op == "rope":
        kv = rng.choice([1, 2, 4, 8, 16])
        heads = kv * rng.choice([1, 2, 4, 8])
        heads = min(heads, 64)
        dim = rng.choice([64, 96, 128, 256])
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        most = 65536 * 40 * 128 * 2 // ((heads + kv) * dim * BYTES[dtype])
        return dict(op="rope", tokens=_log_uniform(rng, 1, min(most, 65536)), heads=heads, kv_heads=kv, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, dim // 4 * 3]), layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "parts"]), span=rng.choice([4096, 32768, 131072]),
                    dtype=dtype, inverse=rng.random() < 0.25, fused_qkv=rng.random() < 0.5)
    if op == "cache":
        kv = rng.choice([1, 2, 4, 8, 16, 32])
        dim = rng.choice([32, 64, 128, 128, 256])
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        most = 8192 * 32 * 128 * 2 // (kv * dim * BYTES[dtype])   # tokens read, in all
        seqs = _log_uniform(rng, 1, min(64, most // 16))
        context = _log_uniform(rng, 1, max(1, most * 3 // (4 * seqs)))
        new = _log_uniform(rng, 1, max(1, min(2048, most // seqs - context)))
        return dict(op="cache", seqs=seqs, new=new, context=context, read_all=rng.random() < 0.7, kv_heads=kv, dim=dim,
                    page=rng.choice([16, 32, 64, 128]), dtype=dtype,
                    rot=rng.choice([dim, dim, dim // 2]) // 16 * 16, layout=rng.choice(["half", "interleaved"]))
    kv = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 2, 4, 4, 8])
    dim = rng.choice([32, 64, 128, 128, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
    seqs = _log_uniform(rng, 1, 64)
    nodes = _log_uniform(rng, 1, 96)
    most = 16 * 32768 * 8 * 128 // (seqs * kv * dim)                                   # by bytes
    most = min(most, 16 * 64 * 32 * 32768 * 128 // (seqs * nodes * kv * group * dim * (4 if dtype == "f32" else 1)))
    context = _log_uniform(rng, 1, max(1, min(262144, most - nodes)))
    return dict(op="tree", seqs=seqs, nodes=nodes, context=context, heads=kv * group, kv_heads=kv, dim=dim,
                page=rng.choice([16, 32, 64, 128]), dtype=dtype, ragged=rng.random() < 0.6, mask=nodes > 1 and rng.random() < 0.8)


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


def _radians(case):
    """Radians per position of each rotated pair, and the magnitude that goes with them."""
    half = case["rot"] // 2
    w = BASE ** (-np.arange(half, dtype=np.float64) / half)
    scaling = case.get("scaling", "none")
    if scaling == "linear":
        return w / 4.0, 1.0
    if scaling == "parts":       # slow pairs interpolated 16 times, fast ones kept, a ramp between 1 and 32 turns per 8192
        turns = 8192 * w / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return w * keep + (w / 16.0) * (1 - keep), 0.1 * math.log(16.0) + 1.0
    return w, 1.0


def _rotary(case, span):
    """What both forms keep for rotary positions: cosines and sines by position, and turns per position in 2^-64."""
    w, scale = _radians(case)
    angle = torch.arange(span, dtype=torch.float64, device=DEV)[:, None] * torch.tensor(w, device=DEV)[None, :]
    turns = [int(round(x / (2 * math.pi) * 2.0**64)) for x in w.tolist()]
    turns = [t - (1 << 64) if t >= 1 << 63 else t for t in turns]
    return {"cos": (angle.cos() * scale).float(), "sin": (angle.sin() * scale).float(),
            "turns": torch.tensor(turns, dtype=torch.int64, device=DEV), "mscale": scale}


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
            top = y.abs().amax(-1)
            q = (y * (7.0 / top)[..., None]).round_().to(torch.int8)
            codes[a:b] = ((q[..., 0::2] & 15) | (q[..., 1::2] << 4)).view(torch.uint8)
            scales[a:b] = top / 7.0 * torch.exp(0.3 * torch.randn(top.shape, generator=g, device=DEV))
        cache[name + "q"], cache[name + "s"] = codes, scales
    return cache


def _spread(n, most, least):
    """n ragged sizes from `least` times `most` up to `most`, which the first has: the same ones for every seed."""
    r = np.random.RandomState(n + most).rand(n)
    return [most] + [int(most * (least + (1 - least) * x)) for x in r[1:]]


def _contexts(case):
    ragged = case.get("ragged", True)
    return _spread(case["seqs"], case["context"], 0.4) if ragged else [case["context"]] * case["seqs"]


def _nodes(case):
    return [max(1, n) for n in _spread(case["seqs"], case["nodes"], 0.5)] if case["ragged"] else [case["nodes"]] * case["seqs"]


def _tables(g, lengths, page):
    """Block tables of sequences whose pages lie anywhere in the pool."""
    need = [-(-n // page) for n in lengths]
    width, total = max(need), sum(need)
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32).cpu()
    table = torch.zeros(len(lengths), width, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table.to(DEV), total


def _prefix(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)


def _outlier_rows(g, tokens, heads, dim, dtype):
    """Normal rows with two large channels in each head."""
    x = torch.randn(tokens, heads, dim, generator=g, device=DEV)
    x[:, :, 3] *= 30.0
    x[:, :, dim - 5] *= 30.0
    return x.to(dtype)


def prepare(case, seed):
    g = _generator(seed)
    dtype = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "rope":
        t, h, kv, d = (case[k] for k in ("tokens", "heads", "kv_heads", "dim"))
        if case["fused_qkv"]:
            rows = torch.randn(t, (h + 2 * kv) * d, generator=g, device=DEV).to(dtype)
            s["q"] = rows[:, :h * d].view(t, h, d)
            s["k"] = rows[:, h * d:(h + kv) * d].view(t, kv, d)
        else:
            s["q"] = torch.randn(t, h, d, generator=g, device=DEV).to(dtype)
            s["k"] = torch.randn(t, kv, d, generator=g, device=DEV).to(dtype)
        s["positions"] = torch.randint(0, case["span"], (t,), generator=g, device=DEV)
        if t > 256:   # prefill: runs of consecutive positions
            s["positions"] = (s["positions"][:1] + torch.arange(t, device=DEV)) % case["span"]
        return {**s, **_rotary(case, case["span"])}
    page, kv, d = case["page"], case["kv_heads"], case["dim"]
    s["rotation"] = torch.tensor(_rotation(d), dtype=torch.float32, device=DEV)
    if case["op"] == "cache":
        contexts, new = _contexts(case), case["new"]
        ends = [c + new for c in contexts]
        s["table"], pages = _tables(g, ends, page)
        s["cache"] = _filled_cache(g, pages, kv, page, d)
        tokens = case["seqs"] * new
        s["k"], s["v"] = (_outlier_rows(g, tokens, kv, d, dtype) for _ in range(2))
        at = torch.cat([torch.arange(c, c + new) for c in contexts]).to(DEV)
        seq = torch.arange(case["seqs"], device=DEV).repeat_interleave(new)
        s["positions"] = at
        s["slots"] = s["table"][seq, at // page].long() * page + at % page
        starts = [0] * len(ends) if case["read_all"] else contexts
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        s["offsets"], s["total"] = _prefix([e - a for a, e in zip(starts, ends)]), sum(ends) - sum(starts)
        if case["rot"]:
            s.update(_rotary(case, max(ends)))
        return s
    contexts, nodes, counts = _contexts(case), case["nodes"], _nodes(case)
    s["table"], pages = _tables(g, [c + n for c, n in zip(contexts, counts)], page)
    s["cache"] = _filled_cache(g, pages, kv, page, d)
    rows = sum(counts)
    s["q"] = (1.5 * torch.randn(rows, case["heads"], d, generator=g, device=DEV)).to(dtype)
    s["contexts"] = torch.tensor(contexts, dtype=torch.int32, device=DEV)
    s["offsets"], s["nodes"], s["longest"] = _prefix(counts), nodes, max(c + n for c, n in zip(contexts, counts))
    s["mask"] = None
    if case["mask"]:
        mask, at = np.zeros((rows, nodes), dtype=bool), 0
        r = torch.rand(rows, generator=g, device=DEV).cpu().numpy()
        for n in counts:
            for i in range(n):
                if i:      # a parent among the nodes before it
                    mask[at + i] = mask[at + int(r[at + i] * i)]
                mask[at + i, i] = True
            at += n
        s["mask"] = torch.tensor(mask, device=DEV)
    # where each padded (sequence, node) takes its row from, and where each row lies in the padded form
    seq = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))
    node = torch.cat([torch.arange(n) for n in counts])
    pad = torch.zeros(len(counts), nodes, dtype=torch.int64)
    pad[seq, node] = torch.arange(rows)
    s["row_of"], s["row_at"] = pad.to(DEV), (seq * nodes + node).to(DEV)
    return s


# ---------------------------------------------------------------- the plain forms, in 32 bits

def _plain_rope(x, cos, sin, rot, layout):
    x = x.float()
    head, rest = x[..., :rot], x[..., rot:]
    cos, sin = cos[:, None, :], sin[:, None, :]
    if layout == "half":
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], -1)
    a, b = head[..., 0::2], head[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), rest], -1)


def _plain_dense(cache, name, pages, rows):
    """Cache rows (page, row of the page) as values in the rotated basis: [..., heads, dim]."""
    b = cache[name + "q"][pages, :, rows]
    q = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    return ((q ^ 8).to(torch.int8) - 8).float() * cache[name + "s"][pages, :, rows][..., None]


def _plain_quantise(x):
    top = x.abs().amax(-1, keepdim=True)
    scale = top / 7.0
    q = torch.where(top > 0, x / scale, torch.zeros_like(x)).round().clamp(-8, 7).to(torch.int8)
    return ((q[..., 0::2] & 15) | (q[..., 1::2] << 4)).view(torch.uint8), scale[..., 0]


def _plain_cache(s):
    case, cache, page = s["case"], s["cache"], s["case"]["page"]
    k, v = s["k"].float(), s["v"].float()
    if case["rot"]:
        k = _plain_rope(k, s["cos"][s["positions"]], s["sin"][s["positions"]], case["rot"], case["layout"])
    to, row = s["slots"] // page, s["slots"] % page
    cache["kq"][to, :, row], cache["ks"][to, :, row] = _plain_quantise(k @ s["rotation"])
    cache["vq"][to, :, row], cache["vs"][to, :, row] = _plain_quantise(v @ s["rotation"])
    i = torch.arange(s["total"], device=DEV)
    seq = torch.searchsorted(s["offsets"], i, right=True) - 1
    at = i - s["offsets"][seq] + s["starts"][seq]
    pages, row = s["table"][seq, at // page].long(), at % page
    dtype = DTYPES[case["dtype"]]
    return {"k": (_plain_dense(cache, "k", pages, row) @ s["rotation"].T).to(dtype),
            "v": (_plain_dense(cache, "v", pages, row) @ s["rotation"].T).to(dtype)}


def _plain_tree(s):
    case, n = s["case"], s["nodes"]
    seqs, heads, kv, d, page = (case[k] for k in ("seqs", "heads", "kv_heads", "dim", "page"))
    group = heads // kv
    at = torch.arange(s["longest"], device=DEV)
    pages, row = s["table"][:, at // page].long(), (at % page).expand(seqs, -1)
    q = (s["q"].float() @ s["rotation"])[s["row_of"]]                          # [seqs, n, heads, d]
    q = q.view(seqs, n, kv, group, d).permute(0, 2, 1, 3, 4).reshape(seqs, kv, n * group, d)
    k = _plain_dense(s["cache"], "k", pages, row).permute(0, 2, 3, 1)          # [seqs, kv, d, longest]
    scores = (q @ k) * d ** -0.5
    node = at[None, :] - s["contexts"][:, None]                                # [seqs, longest]: the node at each place
    if s["mask"] is None:
        seen = node[:, None, :] <= torch.arange(n, device=DEV)[None, :, None]
    else:
        mask = s["mask"][s["row_of"]]                                          # [seqs, n, n]
        seen = (node < 0)[:, None, :] | (torch.gather(mask, 2, node.clamp(0, n - 1)[:, None, :].expand(-1, n, -1)) & (node >= 0)[:, None, :])
    seen = seen & (node < (s["offsets"][1:] - s["offsets"][:-1])[:, None])[:, None, :]
    seen = seen[:, None, :, None, :].expand(-1, kv, -1, group, -1).reshape(seqs, kv, n * group, -1)
    scores = torch.where(seen, scores, -torch.inf)
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    total = p.sum(-1, keepdim=True)
    v = _plain_dense(s["cache"], "v", pages, row).permute(0, 2, 1, 3)          # [seqs, kv, longest, d]
    o = (p @ v) / total @ s["rotation"].T
    o = o.view(seqs, kv, n, group, d).permute(0, 2, 1, 3, 4).reshape(seqs * n, heads, d)
    return o[s["row_at"]].to(DTYPES[case["dtype"]])


def run(s):
    case = s["case"]
    if own:
        import rotational_w4a4_quantization_gb300 as rq
        if case["op"] == "rope":
            q, k = rq.rope(s["q"], s["k"], s["positions"], s["turns"], interleaved=case["layout"] == "interleaved",
                           inverse=case["inverse"], mscale=s["mscale"])
            return {"q": q, "k": k}
        if case["op"] == "cache":
            rq.kv_append(s["k"], s["v"], s["cache"], s["slots"], SEED, FLAGS, positions=s["positions"],
                         turns=s["turns"], interleaved=case["layout"] == "interleaved")
            k, v = rq.kv_read(s["cache"], s["table"], s["starts"], s["offsets"], s["total"], SEED, FLAGS,
                              dtype=DTYPES[case["dtype"]])
            return {"k": k, "v": v}
        return rq.attn_tree(s["q"], s["cache"], s["table"], s["contexts"], s["offsets"], SEED, FLAGS,
                            tree_mask=s["mask"], max_nodes=s["nodes"])
    if case["op"] == "rope":
        cos, sin = s["cos"][s["positions"]], s["sin"][s["positions"]]
        sin = -sin if case["inverse"] else sin
        dtype = DTYPES[case["dtype"]]
        return {"q": _plain_rope(s["q"], cos, sin, case["rot"], case["layout"]).to(dtype),
                "k": _plain_rope(s["k"], cos, sin, case["rot"], case["layout"]).to(dtype)}
    if case["op"] == "cache":
        return _plain_cache(s)
    return _plain_tree(s)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    size = BYTES[case["dtype"]]
    if case["op"] == "rope":
        rows = case["tokens"] * (case["heads"] + case["kv_heads"])
        return {"bytes": 2 * rows * case["dim"] * size + 8 * case["tokens"], "flops": 3 * rows * case["rot"]}
    d, kv, contexts = case["dim"], case["kv_heads"], _contexts(case)
    if case["op"] == "cache":
        new = case["seqs"] * case["new"]
        rows = (2 * new + (sum(contexts) if case["read_all"] else 0)) * 2 * kv
        return {"bytes": rows * (d * size + d // 2 + 4) + 16 * new, "flops": rows * d * (int(math.log2(d)) + 3)}
    counts = _nodes(case)
    seen = sum(n * (c + n) for c, n in zip(contexts, counts))
    return {"bytes": (sum(contexts) + sum(counts)) * kv * (d + 8) + 2 * sum(counts) * case["heads"] * d * size,
            "flops": 4 * seen * case["heads"] * d}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_angles(case, positions):
    w, scale = _radians(case)
    angle = positions.double()[:, None] * torch.tensor(w, device=DEV)[None, :]
    return torch.polar(torch.full_like(angle, scale), angle)        # one complex number per pair


def _exact_rope(x, turn, rot, layout):
    x = x.double()
    head = x[..., :rot]
    if layout == "half":
        z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * turn[:, None, :]
        done = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2)) * turn[:, None, :]
        done = torch.view_as_real(z).flatten(-2)
    return torch.cat([done, x[..., rot:]], -1)


def _exact_rows(codes, scales):
    low = (codes & 15).double()
    high = torch.div(codes, 16, rounding_mode="floor").double()
    q = torch.stack([low, high], -1).flatten(-2)
    return torch.where(q > 7.5, q - 16.0, q) * scales.double()[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        turn = _exact_angles(case, s["positions"])
        turn = turn.conj() if case["inverse"] else turn
        return {name: _exact_rope(s[name], turn, case["rot"], case["layout"]) for name in ("q", "k")}
    r = torch.tensor(_rotation(case["dim"]), device=DEV)
    page, table, cache = case["page"], s["table"].cpu(), s["cache"]
    if case["op"] == "cache":
        new = {"k": s["k"].double(), "v": s["v"].double()}
        if case["rot"]:
            new["k"] = _exact_rope(new["k"], _exact_angles(case, s["positions"]), case["rot"], case["layout"])
        offsets, starts, out = s["offsets"].cpu().tolist(), s["starts"].cpu().tolist(), {"k": [], "v": []}
        for name in ("k", "v"):
            y = new[name] @ r
            step = y.abs().amax(-1, keepdim=True) / 7.0
            y = torch.where(step > 0, (y / step).round().clamp(-8, 7), 0.0) * step.float().double()
            for b in range(case["seqs"]):
                end = starts[b] + offsets[b + 1] - offsets[b]
                used = table[b, :-(-end // page)].long().to(DEV)
                old = _exact_rows(cache[name + "q"][used].transpose(1, 2).flatten(0, 1),
                                  cache[name + "s"][used].transpose(1, 2).flatten(0, 1))[:end]
                old[end - case["new"]:] = y[b * case["new"]:(b + 1) * case["new"]]
                out[name].append(old[starts[b]:] @ r.T)
        return {name: torch.cat(v) for name, v in out.items()}
    offsets, contexts, outs = s["offsets"].cpu().tolist(), s["contexts"].cpu().tolist(), []
    group = case["heads"] // case["kv_heads"]
    for b in range(case["seqs"]):
        rows, c = slice(offsets[b], offsets[b + 1]), contexts[b]
        n = offsets[b + 1] - offsets[b]
        used = table[b, :-(-(c + n) // page)].long().to(DEV)
        seen = torch.ones(n, c + n, dtype=torch.bool, device=DEV)
        seen[:, c:] = torch.ones(n, n, dtype=torch.bool, device=DEV).tril() if s["mask"] is None else s["mask"][rows, :n]
        o = torch.empty(n, case["heads"], case["dim"], dtype=torch.float64, device=DEV)
        for h in range(case["kv_heads"]):
            k = _exact_rows(cache["kq"][used, h].flatten(0, 1), cache["ks"][used, h].flatten())[:c + n] @ r.T
            v = _exact_rows(cache["vq"][used, h].flatten(0, 1), cache["vs"][used, h].flatten())[:c + n] @ r.T
            q = s["q"][rows, h * group:(h + 1) * group].double()
            score = torch.einsum("ngd,td->ngt", q, k) / math.sqrt(case["dim"])
            p = torch.softmax(score.masked_fill(~seen[:, None, :], -math.inf), -1)
            o[:, h * group:(h + 1) * group] = torch.einsum("ngt,td->ngd", p, v)
        outs.append(o)
    return torch.cat(outs)
