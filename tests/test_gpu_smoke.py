"""The smoke run shows the kernels: each of them is launched before the comparisons, which launch many times as many."""
import pytest
import torch

import oracle
import rotational_w4a4_quantization_gb300 as rq
from rotational_w4a4_quantization_gb300 import _binding, prefix_step, tree_step

pytestmark = pytest.mark.gpu


def test_the_operators_come_before_what_they_are_compared_with(monkeypatch):
    import __graft_entry__
    order, sizes = [], []

    def noted(owner, name, label):
        was = getattr(owner, name)

        def call(*args, **kw):
            order.append(label(args))
            return was(*args, **kw)
        monkeypatch.setattr(owner, name, call)

    noted(_binding, "_call", lambda args: args[1])
    for name in ("fwht_quant", "kv_rotate_quant", "w4a4_gemm"):               # these call the library by themselves
        noted(rq, name, lambda args, name=name: "rq_" + name)
    noted(oracle, "fwht_quant", lambda args: "compare")
    for step in (tree_step.TreeStep, prefix_step.PrefixStep):
        noted(step, "error", lambda args: "compare")
    noted(prefix_step, "attn_prefix", lambda args: sizes.append((args[0].shape, args[5].shape, args[1]["kq"].shape)) or "attn_prefix")
    __graft_entry__.smoke()
    before = order[:order.index("compare")]
    for entry in ("rq_fwht_quant", "rq_kv_rotate_quant", "rq_rope", "rq_kv_append", "rq_attn_tree", "rq_kv_plan", "rq_attn_prefix",
                  "rq_w4a16_gemm"):
        assert entry in before, entry
    # the blocks of 256 rows are among them: more than 128 rows to a KV head, and 10 tiles and more for each SM
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert any(q[0] * q[1] // kq[1] // table[0] > 128 and table[0] * kq[1] * -(-table[1] * kq[2] // 128) >= 10 * sms
               for q, table, kq in sizes)
    assert rq.sync_status() == 0
