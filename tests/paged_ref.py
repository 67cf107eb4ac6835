"""Plain 64-bit forms of rotary positions, the paged rotated INT4 cache and tree
attention (test infrastructure; shares no code with the library)."""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle

UNIT = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}   # unit roundoff: half an ulp of 1


def rotation(n: int, seed: int, flags: int) -> torch.Tensor:
    """R as an fp64 matrix: row i is the rotation of the i-th unit vector."""
    return torch.from_numpy(oracle.rotate(np.eye(n), seed, flags))


def turn(x, positions, turns, interleaved, mscale=1.0, inverse=False):
    """Rotary positions of x [T][H][D] in fp64, from the integer frequencies (exact angles)."""
    x = x.double()
    rot = 2 * len(turns)
    w = [int(t) % (1 << 64) for t in turns.tolist()]
    frac = [[((int(p) * f) % (1 << 64)) / 2.0**64 for f in w] for p in positions.tolist()]
    ang = torch.tensor(frac, dtype=torch.float64).reshape(len(positions), len(w)).to(x.device) * (2 * math.pi)
    c, s = ang.cos()[:, None, :] * mscale, ang.sin()[:, None, :] * mscale
    if inverse:
        s = -s
    y = x.clone()
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(0, rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = a * s + b * c
    return y


def decode(codes, scales):
    """Packed codes [..., D/2] and scales [...] -> fp64 values [..., D]."""
    b = codes.to(torch.int64)
    n = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    return torch.where(n >= 8, n - 16, n).double() * scales.double()[..., None]


def places(table, page, b, count):
    """(page, row) of the first `count` tokens of sequence b."""
    t = torch.arange(count)
    return table[b].cpu().long()[t // page], t % page


def attention(q, cache, table, contexts, offsets, seed, flags, scale, mask=None, rotated=False, pages_ok=None):
    """Tree attention in fp64.  Returns (out, spread, delta): spread is sum_t p_t |v_t| (rotated basis) and delta the
    root of the largest sum_d (q_d k_td)^2 * scale, the size that rounding the rotated queries acts on."""
    q = q.double()
    N, Hq, D = q.shape
    dev = q.device
    kq, ks, vq, vs = (cache[n] for n in ("kq", "ks", "vq", "vs"))
    H, page = kq.shape[1], kq.shape[2]
    R = rotation(D, seed, flags & 1).to(dev)
    out, spread = torch.zeros(N, Hq, D, dtype=torch.float64, device=dev), torch.zeros(N, Hq, D, dtype=torch.float64, device=dev)
    delta = torch.zeros(N, Hq, dtype=torch.float64, device=dev)
    for b in range(table.shape[0]):
        r0, r1, c = int(offsets[b]), int(offsets[b + 1]), int(contexts[b])
        n = r1 - r0
        L = min(c + n, table.shape[1] * page)
        if n == 0 or L == 0:
            continue
        pg, row = places(table, page, b, L)
        good = (pg >= 0) & (pg < kq.shape[0])
        pg = torch.where(good, pg, 0)
        seen = torch.zeros(n, L, dtype=torch.bool)
        seen[:, :min(c, L)] = True
        for i in range(n):
            for j in range(n):
                if c + j < L and (bool(mask[r0 + i, j]) if mask is not None else j <= i):
                    seen[i, c + j] = True
        seen &= good[None, :]
        seen = seen.to(dev)
        for h in range(Hq):
            kv = h // (Hq // H)
            k = decode(kq[pg, kv, row], ks[pg, kv, row]).to(dev)
            v = decode(vq[pg, kv, row], vs[pg, kv, row]).to(dev)
            qr = q[r0:r1, h] @ R
            for i in range(n):
                idx = seen[i].nonzero()[:, 0]
                if len(idx) == 0:
                    continue
                s = (k[idx] @ qr[i]) * scale
                p = torch.softmax(s, 0)
                o = p @ v[idx]
                out[r0 + i, h] = o if rotated else o @ R.T
                spread[r0 + i, h] = p @ v[idx].abs()
                delta[r0 + i, h] = (k[idx] ** 2 @ qr[i] ** 2).max().sqrt() * abs(scale)
    return out, spread, delta


def tree_mask(counts, generator, width=None):
    """Ancestor masks of random trees, one after the other: bool [sum(counts)][width]."""
    width = width or max(counts)
    m = torch.zeros(sum(counts), width, dtype=torch.bool)
    at = 0
    for n in counts:
        for i in range(n):
            if i:
                parent = int(torch.randint(0, i, (1,), generator=generator))
                m[at + i] = m[at + parent]
            m[at + i, i] = True
        at += n
    return m


def attention_blocks(q, cache, table, contexts, offsets, seed, flags, scale, mask=None):
    """attention() for larger cases: a sequence at a time, all heads and nodes at once.  Needs valid pages and at least
    one visible token in every row.  Returns (out, spread, delta) as attention() does."""
    q = q.double()
    N, Hq, D = q.shape
    H, page = cache["kq"].shape[1], cache["kq"].shape[2]
    R = rotation(D, seed, flags & 1).to(q.device)
    out, spread, delta = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(N, Hq, dtype=torch.float64, device=q.device)
    for b in range(table.shape[0]):
        r0, r1, c = int(offsets[b]), int(offsets[b + 1]), int(contexts[b])
        n, L = r1 - r0, c + r1 - r0
        if n == 0:
            continue
        pg, row = (x.to(q.device) for x in places(table, page, b, L))
        k = decode(cache["kq"][pg, :, row], cache["ks"][pg, :, row]).transpose(0, 1)      # [H][L][D]
        v = decode(cache["vq"][pg, :, row], cache["vs"][pg, :, row]).transpose(0, 1)
        seen = torch.ones(n, L, dtype=torch.bool, device=q.device)
        seen[:, c:] = torch.ones(n, n, dtype=torch.bool).tril().to(q.device) if mask is None else mask[r0:r1, :n].to(q.device)
        qr = (q[r0:r1] @ R).view(n, H, Hq // H, D)
        s = torch.einsum("nhgd,hld->nhgl", qr, k) * scale
        p = torch.softmax(s.masked_fill(~seen[:, None, None, :], -math.inf), -1)
        out[r0:r1] = (torch.einsum("nhgl,hld->nhgd", p, v) @ R.T).reshape(n, Hq, D)
        spread[r0:r1] = torch.einsum("nhgl,hld->nhgd", p, v.abs()).reshape(n, Hq, D)
        delta[r0:r1] = (torch.einsum("nhgd,hld->nhgl", qr ** 2, k ** 2).amax(-1).sqrt() * abs(scale)).reshape(n, Hq)
    return out, spread, delta
