"""Decode steps of requests that share a prompt, on the paged rotated INT4 cache.

    python -m rotational_w4a4_quantization_gb300.prefix_step --prefix 8192 --own 256 --groups 2 --seqs 64

Requests come in groups with one long prompt each, which the cache holds once; what a request
has had since lies on pages of its own.  A step of one attention layer and its output
projection is:

1. :func:`kv_plan` gives each request's new token its page and slot;
2. :func:`kv_append` writes the tokens' keys, turned to their positions, and values there;
3. :func:`rope` turns their queries;
4. :func:`attn_prefix` attends to the group's prompt, read for blocks of all its rows, and to
   the request's own tokens, and leaves the rows in the rotated basis;
5. :func:`w4a16_gemm` multiplies them, 64 at a time, with the output weights, into which the
   heads' rotation is folded (one scale per channel and head).

Nothing of it waits for the host, so a step can be captured in a CUDA graph and replayed: the
lengths and the free list's head advance on the device.  Prints the step's time and how far
its output lies from a 64-bit computation over the same rows.  Inputs are random.
"""
from __future__ import annotations

import argparse

import torch

from . import (RQ_ATTN_ROTATED_OUT, RQ_GROUP_SCALES, RQ_KV_ROTATED_OUT, RQ_SIGNS_FIRST, attn_prefix,
               attn_prefix_workspace, fwht_quant, kv_append, kv_cache, kv_plan, kv_read, rope, rope_turns, sync_status,
               w4a16_gemm)

SEED = 0x5EED
DIM = 128              # a head is a group of 128 weights


class PrefixStep:
    """The cache, the page tables, the folded output weights and the buffers of the step."""

    def __init__(self, seqs: int, groups: int, prefix: int, own: int, heads: int, kv_heads: int, page: int, hidden: int,
                 steps: int = 64, dtype=torch.bfloat16, device="cuda", seed: int = 1):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.prefix, self.page = seqs, prefix, page
        i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).to(device)
        rand = lambda *shape: torch.randn(*shape, generator=g).to(dtype).to(device)
        wide, own_wide = -(-prefix // page), -(-(own + steps) // page)
        pages = groups * wide + seqs * own_wide
        self.cache = kv_cache(pages, kv_heads, DIM, page, device)
        self.free = torch.randperm(pages, generator=g).to(torch.int32).to(device)
        self.turns, self.mscale = rope_turns(DIM, device=device)
        self.groups = i32([seqs * i // groups for i in range(groups + 1)])
        self.prefix_lens = i32([prefix] * groups)
        self.base = i32([prefix] * seqs)
        self.offsets = i32(range(seqs + 1))
        self.prefix_table = torch.full((groups, max(1, wide)), -1, dtype=torch.int32, device=device)
        self.table = torch.full((seqs, own_wide), -1, dtype=torch.int32, device=device)
        # the prompts, then what each request has had since
        none = lambda n: torch.zeros(n, dtype=torch.int32, device=device)
        _, slots, at, self.head = kv_plan(none(groups), self.prefix_lens, self.prefix_table, self.free, groups * prefix, page)
        self._write(rand(groups * prefix, kv_heads, DIM), rand(groups * prefix, kv_heads, DIM), slots, at)
        self.contexts = i32([own * (b % 3 + 1) // 3 for b in range(seqs)])
        total = int(self.contexts.sum())
        _, slots, at, self.head = kv_plan(none(seqs), self.contexts, self.table, self.free, total, page, head=self.head,
                                          base=self.base)
        self._write(rand(total, kv_heads, DIM), rand(total, kv_heads, DIM), slots, at)
        # W^T, one row per output channel and head: R folded in, a scale for each
        weights = 0.02 * torch.randn(hidden * heads, DIM, generator=g).to(device)
        codes, scales = fwht_quant(weights, SEED, RQ_SIGNS_FIRST | RQ_GROUP_SCALES)
        self.w, self.w_scales = codes.view(hidden, heads * DIM // 2), scales.view(hidden, heads)
        self.q, self.k, self.v = rand(seqs, heads, DIM), rand(seqs, kv_heads, DIM), rand(seqs, kv_heads, DIM)
        self.one = torch.ones(seqs, dtype=torch.int32, device=device)
        self.rows = torch.empty_like(self.q)
        self.y = torch.empty(seqs, hidden, dtype=dtype, device=device)
        self.plan = (torch.empty(seqs + 1, dtype=torch.int32, device=device), torch.empty(seqs, dtype=torch.int64, device=device),
                     torch.empty(seqs, dtype=torch.int64, device=device), torch.empty_like(self.head))
        self.workspace = torch.empty(attn_prefix_workspace(seqs, heads, DIM), dtype=torch.uint8, device=device)

    def _write(self, k, v, slots, at):
        kv_append(k, v, self.cache, slots, SEED, positions=at, turns=self.turns, mscale=self.mscale)

    def step(self):
        """One token of every request: (turned queries, attention rows in the rotated basis, their projection)."""
        _, slots, at, head = kv_plan(self.contexts, self.one, self.table, self.free, self.seqs, self.page, head=self.head,
                                     base=self.base, out=self.plan)
        self._write(self.k, self.v, slots, at)
        q, _ = rope(self.q, None, at, self.turns, mscale=self.mscale)
        attn_prefix(q, self.cache, self.table, self.contexts, self.offsets, self.prefix_table, self.prefix_lens, self.groups,
                    SEED, RQ_SIGNS_FIRST | RQ_ATTN_ROTATED_OUT, max_nodes=1, out=self.rows, workspace=self.workspace)
        for at in range(0, self.seqs, 64):               # as many rows as a product takes
            w4a16_gemm(self.rows[at:at + 64].flatten(1), self.w, self.w_scales, out=self.y[at:at + 64])
        self.contexts += self.one
        self.head.copy_(head)
        return q, self.rows, self.y

    def error(self, q, y) -> float:
        """Largest relative distance of an output row from 64 bits over the cache's rows (after a step)."""
        lens, prefixes, groups = self.contexts.tolist(), self.prefix_lens.tolist(), self.groups.tolist()
        H = self.cache["kq"].shape[1]

        def rows(table, counts):         # dense, in the rotated basis, as the weights are
            offsets = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32)
            k, v = kv_read(self.cache, table, None, offsets.to(q.device), sum(counts), SEED, RQ_SIGNS_FIRST | RQ_KV_ROTATED_OUT,
                           dtype=torch.float32)
            return k.split(counts), v.split(counts)

        pk, pv = rows(self.prefix_table, prefixes)
        ok, ov = rows(self.table, lens)
        heads = q.shape[1]
        turned = fwht_quant(q.reshape(-1, DIM).float(), SEED, RQ_SIGNS_FIRST, want_y=True)[2].view(q.shape).double()
        b = self.w.to(torch.int64)
        codes = torch.stack([b & 15, b >> 4], -1).flatten(1)
        w = torch.where(codes >= 8, codes - 16, codes).double().view(-1, heads, DIM) * self.w_scales.double()[..., None]
        worst = 0.0
        for i, (first, last) in enumerate(zip(groups, groups[1:])):
            for r in range(first, last):
                k, v = (torch.cat(x).double() for x in ((pk[i], ok[r]), (pv[i], ov[r])))
                s = torch.einsum("hgd,thd->hgt", turned[r].view(H, heads // H, DIM), k) * DIM ** -0.5
                o = torch.einsum("hgt,thd->hgd", torch.softmax(s, -1), v).reshape(heads, DIM)
                want = torch.einsum("hd,nhd->n", o, w)
                worst = max(worst, float((y[r].double() - want).norm() / want.norm()))
        return worst


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--seqs", type=int, default=64)
    ap.add_argument("--groups", type=int, default=2)
    ap.add_argument("--prefix", type=int, default=8192)
    ap.add_argument("--own", type=int, default=256)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--page", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    work = PrefixStep(a.seqs, a.groups, a.prefix, a.own, a.heads, a.kv_heads, a.page, a.hidden, a.steps + 3)
    for _ in range(3):
        work.step()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(a.steps):
        q, _, y = work.step()
    end.record()
    torch.cuda.synchronize()
    err = work.error(q, y)
    if sync_status():
        raise RuntimeError("a kernel's wait ran out")
    print(f"{a.seqs} requests in {a.groups} groups, prompts of {a.prefix}, {a.heads}/{a.kv_heads} heads x {DIM}: "
          f"{begin.elapsed_time(end) / a.steps * 1e3:.1f} us a step, largest relative error {err:.1e}")


if __name__ == "__main__":
    main()
