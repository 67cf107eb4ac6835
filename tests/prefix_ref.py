"""Plain forms of block tables from lengths, shared-prefix attention and products with 4-bit weights (test
infrastructure; shares no code with the library)."""
from __future__ import annotations

import torch

import paged_ref


def plan(contexts, new, table, free, total, page, head=0, base=None):
    """Request by request, token by token: (offsets, slots, positions, head') and the table, as lists."""
    table = [list(r) for r in table]
    slots, positions, offsets, at = [-1] * total, [0] * total, [0], head
    width = len(table[0]) if table else 0
    for b, (c, n) in enumerate(zip(contexts, new)):
        c, n = max(0, c), max(0, n)
        kept, need = min(-(-c // page), width), min(-(-(c + n) // page), width)
        for j in range(kept, width):
            table[b][j] = -1
            if j < need:
                table[b][j] = free[at] if 0 <= at < len(free) else -1
                at += 1
        for i in range(n):
            row, place = offsets[-1] + i, c + i
            if row >= total:
                break
            number = table[b][place // page] if place // page < width else -1
            slots[row] = number * page + place % page if number >= 0 else -1
            positions[row] = place + (0 if base is None else base[b])
        offsets.append(offsets[-1] + n)
    return offsets, slots, positions, at, table


def joined(cache, table, contexts, counts, prefix_table, prefix_lens, groups):
    """A cache with pages of one token and tables that name each sequence's prefix and own tokens one after the other:
    (cache, table, contexts) for the plain forms of tree attention.  A page number outside the cache stays one."""
    pages, H, page, _ = cache["kq"].shape
    flat = {n: t.transpose(1, 2).flatten(0, 1).unsqueeze(2) for n, t in cache.items()}        # [pages * page][H][1]..

    def places(row, n):
        n = min(max(0, n), len(row) * page)
        return [row[t // page] * page + t % page if 0 <= row[t // page] < pages else -1 for t in range(n)]

    rows, ctx = [], []
    prefix_of = {}
    for g in range(len(prefix_lens)):
        for b in range(int(groups[g]), int(groups[g + 1])):
            prefix_of[b] = g
    table, prefix_table = table.tolist(), prefix_table.tolist()
    for b, (c, n) in enumerate(zip(contexts, counts)):
        g = prefix_of.get(b)
        before = [] if g is None else places(prefix_table[g], int(prefix_lens[g]))
        rows.append(before + places(table[b], c + n))
        ctx.append(len(before) + min(max(0, c), len(table[b]) * page))
    out = torch.full((len(rows), max(1, max(map(len, rows)))), -1, dtype=torch.int32)
    for b, r in enumerate(rows):
        out[b, :len(r)] = torch.tensor(r, dtype=torch.int32)
    return flat, out, torch.tensor(ctx, dtype=torch.int32)


def weights(codes, scales):
    """Packed codes [N][K/2] and scales [N] or [N][K/128] as fp64 [N][K]."""
    n = codes.shape[0]
    groups = scales.reshape(n, -1)
    return paged_ref.decode(codes.view(n, groups.shape[1], -1), groups).flatten(1)
