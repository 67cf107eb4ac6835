"""A prefix so long that the first pass of shared-prefix attention takes longer than the kernels' limit on their waits
(4e9 cycles, about 2 s), while blocks of the second already stand beside it."""
import pytest
import torch

import rotational_w4a4_quantization_gb300 as rq
from test_gpu_paged import DEV, SEED, _built, _status, dev_cache, filled_cache, randn  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_first_pass_beyond_the_limit_of_waits():
    """The prefix names the same pages over and over: first one whose key scales are so far apart that it goes token by
    token, then one that does not.  Blocks that have the latter end at less than half of the time and leave their place to
    the second pass, whose units are several to a block.  The prefix's codes are 0, so that each of its tokens has weight
    1 and adds nothing; own scores spread so far that the own tokens' sum is of that size.  What may be off: the queries'
    rounding to fp16, 2^-12 of scores below 30 (7e-3), the weights' and their sum's, 2^-12 each, and the output's, 2^-8."""
    H, seqs, D, page, own = 16, 60, 64, 256, 1000
    each = -(-own // page)
    cache = filled_cache(2 + seqs * each, H, page, D, 600)
    cache["kq"][:2], cache["vq"][:2], cache["ks"][:2], cache["vs"][:2] = 0, 0, 1.0, 1.0
    cache["ks"][0, :, ::2] = 2.0**-20
    cache = dev_cache(cache)
    q = randn(seqs, H, D, seed=601, dtype=torch.bfloat16).to(DEV)
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).to(DEV)
    table = i32(range(2, 2 + seqs * each)).view(seqs, each)
    contexts, offsets, groups = i32([own - 1] * seqs), i32(range(seqs + 1)), i32([0, seqs])

    flags = rq.RQ_SIGNS_FIRST | rq.RQ_ATTN_ROTATED_OUT
    k, v = rq.kv_read(cache, table, None, i32([own * b for b in range(seqs + 1)]), own * seqs, SEED,
                      rq.RQ_SIGNS_FIRST | rq.RQ_KV_ROTATED_OUT, dtype=torch.float32)
    turned = rq.fwht_quant(q.float().view(-1, D), SEED, rq.RQ_SIGNS_FIRST, want_y=True)[2].view(seqs, H, D).double()
    scores = torch.einsum("bhd,bthd->bht", turned, k.view(seqs, own, H, D).double())
    scale = 3.0 / float(scores.std())

    def call(pages, first=0):
        prefix = torch.full((1, 2 * pages), first, dtype=torch.int32, device=DEV)
        prefix[0, pages:] = 1
        return lambda: rq.attn_prefix(q, cache, table, contexts, offsets, prefix, i32([2 * pages * page]), groups, SEED, flags,
                                      max_nodes=1, softmax_scale=scale)

    def seconds(run):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        got = run()
        end.record()
        torch.cuda.synchronize()
        return begin.elapsed_time(end) * 1e-3, got

    few = 1 << 14
    seconds(call(few))
    slow, fast = seconds(call(few))[0], seconds(call(few, 1))[0]
    pages = min((1 << 22) - 1, int(few * 2.8 / (slow - fast)))
    took, got = seconds(call(pages))
    assert rq.sync_status() == 0
    assert took * (1 - fast / slow) > 2.5           # between the ends of the first blocks and of the last: else it shows nothing
    e = torch.exp(scores * scale)
    want = torch.einsum("bht,bthd->bhd", e, v.view(seqs, own, H, D).double()) / (e.sum(-1) + 2.0 * pages * page)[..., None]
    err = ((got.double() - want).norm(dim=-1) / want.norm(dim=-1)).max()
    assert float((scores * scale).abs().max()) < 30 and err < 7.4e-3 + 2.0**-11 + 2.0**-8, float(err)
