"""One verification step of speculative decoding on the paged rotated INT4 cache.

    python -m rotational_w4a4_quantization_gb300.tree_step --context 4096 --nodes 32 --seqs 8

A batch of sequences has its prompts in the cache; each drafts a tree of tokens.  The step
of one attention layer is:

1. :func:`kv_append` writes the nodes' keys, turned to their positions (context + depth),
   and values behind each context;
2. :func:`rope` turns their queries;
3. :func:`attn_tree` attends from every node to the context and the node's ancestors;
4. the accepted path's keys and values are written again, one after the other (a path's
   nodes need not be neighbours), which leaves the cache as a plain decode expects it.

Prints the step's time and how far its output lies from a 64-bit attention over the rows
that :func:`kv_read` returns.  Inputs are random: no weights are needed to run it.
"""
from __future__ import annotations

import argparse

import torch

from . import attn_tree, kv_append, kv_cache, kv_plan, kv_read, rope, rope_turns, sync_status

SEED = 0x5EED


def drafted_tree(nodes: int, generator: torch.Generator):
    """A random tree over one root: (mask [nodes][nodes] of ancestors and self, depth [nodes])."""
    mask, depth = torch.eye(nodes, dtype=torch.bool), torch.zeros(nodes, dtype=torch.int64)
    for i in range(1, nodes):
        parent = int(torch.randint(max(0, i - 4), i, (1,), generator=generator))
        mask[i] |= mask[parent]
        depth[i] = depth[parent] + 1
    return mask, depth


class TreeStep:
    """The cache, the page table and the buffers of the step, laid out once and used for every layer call."""

    def __init__(self, seqs: int, context: int, nodes: int, heads: int, kv_heads: int, dim: int, page: int,
                 dtype=torch.bfloat16, device="cuda", seed: int = 1):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.context, self.nodes, self.page = seqs, context, nodes, page
        width = (context + nodes + page - 1) // page
        self.cache = kv_cache(seqs * width, kv_heads, dim, page, device)
        free = torch.randperm(seqs * width, generator=g).to(torch.int32).to(device)
        self.turns, self.mscale = rope_turns(dim, device=device)
        mask, depth = zip(*(drafted_tree(nodes, g) for _ in range(seqs)))
        self.mask = torch.cat(mask).to(device)
        self.depth = torch.stack(depth).to(device)
        self.contexts = torch.full((seqs,), context, dtype=torch.int32, device=device)
        self.offsets = torch.arange(seqs + 1, dtype=torch.int32, device=device) * nodes
        rand = lambda rows, h: torch.randn(rows, h, dim, generator=g).to(dtype).to(device)
        self.q = rand(seqs * nodes, heads)
        self.k, self.v = rand(seqs * nodes, kv_heads), rand(seqs * nodes, kv_heads)
        # pages for the prompts, then for the nodes behind them
        self.table = torch.full((seqs, width), -1, dtype=torch.int32, device=device)
        _, slots, place, head = kv_plan(torch.zeros_like(self.contexts), self.contexts, self.table, free, seqs * context, page)
        kv_append(rand(seqs * context, kv_heads), rand(seqs * context, kv_heads), self.cache, slots, SEED,
                  positions=place, turns=self.turns, mscale=self.mscale)
        _, self.node_slots, _, _ = kv_plan(self.contexts, torch.full_like(self.contexts, nodes), self.table, free,
                                           seqs * nodes, page, head=head)
        self.positions = (context + self.depth).flatten()
        self.out = torch.empty_like(self.q)

    def slots(self, place):
        """Slots of the places [seqs][n] in the sequences: page * page_size + row."""
        return (self.table.gather(1, place // self.page).long() * self.page + place % self.page).flatten()

    def attend(self):
        """Steps 1 to 3: the nodes enter the cache, their queries turn and attend."""
        kv_append(self.k, self.v, self.cache, self.node_slots, SEED, positions=self.positions, turns=self.turns,
                  mscale=self.mscale)
        q, _ = rope(self.q, None, self.positions, self.turns, mscale=self.mscale)
        attn_tree(q, self.cache, self.table, self.contexts, self.offsets, SEED, tree_mask=self.mask, out=self.out)
        return q, self.out

    def accept(self, path):
        """Step 4: path [seqs][n] of node numbers, root first, becomes the sequences' next n tokens."""
        rows = (path + self.nodes * torch.arange(self.seqs, device=path.device)[:, None]).flatten()
        place = self.context + torch.arange(path.shape[1], device=path.device).repeat(self.seqs, 1)
        kv_append(self.k[rows], self.v[rows], self.cache, self.slots(place), SEED, positions=place.flatten(),
                  turns=self.turns, mscale=self.mscale)

    def error(self, q, out) -> float:
        """Largest relative distance of an output row from the 64-bit attention over the cache's rows."""
        rows = self.context + self.nodes
        offsets = torch.arange(self.seqs + 1, dtype=torch.int32, device=q.device) * rows
        kd, vd = kv_read(self.cache, self.table, None, offsets, self.seqs * rows, SEED, dtype=torch.float32)
        group, worst = q.shape[1] // kd.shape[1], 0.0
        for b in range(self.seqs):
            own = slice(b * self.nodes, (b + 1) * self.nodes)
            seen = torch.cat([torch.ones(self.nodes, self.context, dtype=torch.bool, device=q.device), self.mask[own]], 1)
            for h in range(q.shape[1]):
                kk, vv = (x[b * rows:(b + 1) * rows, h // group].double() for x in (kd, vd))
                s = (q[own, h].double() @ kk.T) * q.shape[-1] ** -0.5
                want = torch.softmax(s.masked_fill(~seen, float("-inf")), -1) @ vv
                worst = max(worst, float(((out[own, h].double() - want).norm(dim=-1) / want.norm(dim=-1)).max()))
        return worst


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--seqs", type=int, default=8)
    ap.add_argument("--context", type=int, default=4096)
    ap.add_argument("--nodes", type=int, default=32)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--dim", type=int, default=128)
    ap.add_argument("--page", type=int, default=64)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    step = TreeStep(a.seqs, a.context, a.nodes, a.heads, a.kv_heads, a.dim, a.page)
    for _ in range(3):
        q, out = step.attend()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(a.steps):
        step.attend()
    end.record()
    torch.cuda.synchronize()
    err = step.error(q, out)
    step.accept(torch.zeros(a.seqs, 1, dtype=torch.int64, device=q.device))
    if sync_status():
        raise RuntimeError("a kernel's wait ran out")
    print(f"{a.seqs} sequences of {a.context}, {a.nodes} drafted tokens each, {a.heads}/{a.kv_heads} heads x {a.dim}: "
          f"{begin.elapsed_time(end) / a.steps * 1e3:.1f} us a step, largest relative error {err:.1e}")


if __name__ == "__main__":
    main()
