"""Host-side checks of the rotary, paged-cache and tree-attention entry points: bad
arguments are refused before anything is enqueued (these calls never touch a GPU)."""
import ctypes
import math

import pytest
import torch

import rotational_w4a4_quantization_gb300 as rq
from rotational_w4a4_quantization_gb300 import build as rq_build

A16, A8, A4, A2, A1 = (ctypes.c_void_p(x) for x in (0x10000, 0x10008, 0x10004, 0x10002, 0x10001))
NULL = None


@pytest.fixture(scope="module")
def lib():
    rq_build.build()
    return rq.load_library()


def rope(lib, q=A16, qh=4, qt=512, qhs=128, qo=A16, k=A16, kh=2, ko=A16, dt=1, T=4, D=128, rot=128, pos=A16, turns=A16,
         flags=0):
    return lib.rq_rope(q, qh, qt, qhs, qo, 512, 128, k, kh, 256, 128, ko, 256, 128, dt, T, D, rot, pos, turns, 1.0, flags, NULL)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), 1),
    (dict(qh=-1), 1),
    (dict(D=0), 1),
    (dict(rot=0), 1),
    (dict(rot=130), 1),               # more than the head
    (dict(rot=63), 1),                # odd
    (dict(flags=1), 1),
    (dict(dt=3), 2),                  # int32 rows
    (dict(D=258, rot=64), 2),
    (dict(D=127, rot=64), 2),         # odd head
    (dict(qh=4096, kh=1), 2),
    (dict(q=NULL), 1),
    (dict(ko=NULL), 1),
    (dict(pos=NULL), 1),
    (dict(turns=NULL), 1),
    (dict(q=A1), 3),                  # not an element boundary
    (dict(dt=0, k=A2), 3),
    (dict(pos=A4), 3),                # int64 entries
    (dict(T=0, q=NULL), 0),
    (dict(qh=0, kh=0, q=NULL, k=NULL), 0),
])
def test_rope_argument_checks(lib, kw, expect):
    assert rope(lib, **kw) == expect


def append(lib, k=A16, kt=1024, v=A16, dt=1, T=4, H=8, D=128, slots=A16, pos=NULL, turns=NULL, rot=0, flags=1, kq=A16,
           ks=A16, vq=A16, vs=A16, pages=4, page=64):
    return lib.rq_kv_append(k, kt, 128, v, 1024, 128, dt, T, H, D, slots, pos, turns, rot, 1.0, 7, flags, kq, ks, vq, vs,
                            pages, page, NULL)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), 1),
    (dict(H=0), 1),
    (dict(pages=-1), 1),
    (dict(page=0), 1),
    (dict(flags=2), 1),
    (dict(dt=3), 2),
    (dict(D=96), 2),
    (dict(D=512), 2),
    (dict(page=8), 2),
    (dict(page=48), 2),
    (dict(page=512), 2),
    (dict(H=5000), 2),
    (dict(kq=NULL), 1),
    (dict(vs=NULL), 1),
    (dict(ks=A4), 3),
    (dict(k=NULL), 1),
    (dict(slots=NULL), 1),
    (dict(slots=A4), 3),
    (dict(k=A8), 3),
    (dict(kt=1028), 3),               # 2056-byte token stride
    (dict(turns=A16, rot=128), 1),    # turns without positions
    (dict(turns=A16, pos=A16, rot=0), 1),
    (dict(turns=A16, pos=A16, rot=136), 1),
    (dict(turns=A16, pos=A16, rot=72), 2),             # half layout: multiples of 16
    (dict(turns=A16, pos=A16, rot=72, flags=5, T=0), 0),   # interleaved: of 8
    (dict(turns=A16, pos=A16, rot=68, flags=5), 2),
    (dict(T=0, k=NULL, slots=NULL), 0),
])
def test_append_argument_checks(lib, kw, expect):
    assert append(lib, **kw) == expect


def read(lib, kq=A16, vs=A16, pages=4, H=8, page=64, D=128, table=A16, W=2, starts=NULL, offsets=A16, B=2, total=10,
         flags=1, ko=A16, vo=A16, dt=1):
    return lib.rq_kv_read(kq, A16, A16, vs, pages, H, page, D, table, W, starts, offsets, B, total, 7, flags, ko, vo, dt, NULL)


@pytest.mark.parametrize("kw,expect", [
    (dict(total=-1), 1),
    (dict(B=-1), 1),
    (dict(W=-1), 1),
    (dict(flags=4), 1),
    (dict(dt=3), 2),
    (dict(D=48), 2),
    (dict(page=24), 2),
    (dict(kq=NULL), 1),
    (dict(table=NULL), 1),
    (dict(offsets=NULL), 1),
    (dict(vo=NULL), 1),
    (dict(ko=A8), 3),
    (dict(starts=A2), 3),
    (dict(total=0, table=NULL), 0),
    (dict(B=0, table=NULL), 0),
])
def test_read_argument_checks(lib, kw, expect):
    assert read(lib, **kw) == expect


def tree(lib, q=A16, qt=4096, dt=1, N=8, Hq=32, D=128, kq=A16, pages=4, H=8, page=64, table=A16, W=2, ctx=A16, off=A16,
         B=2, nodes=4, mask=NULL, ms=0, flags=1, out=A16, ws=A16, wb=1 << 40):
    return lib.rq_attn_tree(q, qt, 128, dt, N, Hq, D, kq, A16, A16, A16, pages, H, page, table, W, ctx, off, B, nodes, mask, ms,
                            7, flags, 0.088, out, ws, wb, NULL)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), 1),
    (dict(Hq=0), 1),
    (dict(B=-1), 1),
    (dict(nodes=-1), 1),
    (dict(flags=4), 1),
    (dict(dt=3), 2),
    (dict(D=96), 2),
    (dict(page=8), 2),
    (dict(Hq=30), 1),                 # does not divide over the KV heads
    (dict(mask=A16, ms=3), 1),        # narrower than max_nodes
    (dict(pages=1 << 24, page=64), 2),        # 2^33 rows
    (dict(W=1 << 26), 2),
    (dict(kq=NULL), 1),
    (dict(q=NULL), 1),
    (dict(table=NULL), 1),
    (dict(W=0), 1),
    (dict(out=NULL), 1),
    (dict(ws=NULL), 1),
    (dict(wb=-1), 1),
    (dict(q=A8), 3),
    (dict(out=A8), 3),
    (dict(qt=4100), 3),
    (dict(ctx=A2), 3),
    (dict(N=0, q=NULL), 0),
    (dict(B=0, q=NULL), 0),
    (dict(nodes=0, q=NULL), 0),
])
def test_tree_argument_checks(lib, kw, expect):
    assert tree(lib, **kw) == expect


# ---- the binding, on CPU tensors: checks come before the device check ----

def _cache(pages=2, H=2, page=16, D=64):
    return rq.kv_cache(pages, H, D, page, device="cpu")


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def test_binding_refuses_rope(lib):
    turns, _ = rq.rope_turns(64, device="cpu")
    x, pos = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int64)
    for kw, match in [
        (dict(q=None, k=None), "both be None"),
        (dict(q=x[0]), "must be \\[tokens\\]"),
        (dict(q=x.transpose(1, 2)), "unit stride"),
        (dict(q=x.double()), "float32, bfloat16 or float16"),
        (dict(k=x.half()), "k: expected dtype"),
        (dict(k=x[:2]), "expected 3 tokens"),
        (dict(k=torch.zeros(3, 2, 32)), "one head_dim"),
        (dict(positions=pos.int()), "positions must be"),
        (dict(positions=pos[:2]), "positions must be"),
        (dict(turns=turns.float()), "turns must be"),
        (dict(turns=torch.zeros(33, dtype=torch.int64)), "rotate 66 of 64"),
        (dict(out=(torch.zeros(3, 1, 64), None)), "out \\(q\\): expected shape"),
        (dict(), "CUDA"),
    ]:
        args = dict(q=x, k=x, positions=pos, turns=turns, out=None) | kw
        with pytest.raises(ValueError, match=match):
            rq.rope(args["q"], args["k"], args["positions"], args["turns"], out=args["out"])


def test_binding_refuses_rope_turns():
    for kw, match in [(dict(rot_dim=7), "even"), (dict(rot_dim=8, scaling="cubic"), "unknown scaling"),
                      (dict(rot_dim=8, factor=0.0), "positive"), (dict(rot_dim=2, scaling="base"), "rot_dim >= 4"),
                      (dict(rot_dim=8, fast=1.0, slow=2.0), "fast above slow")]:
        with pytest.raises(ValueError, match=match):
            rq.rope_turns(device="cpu", **kw)
    turns, m = rq.rope_turns(4, 10000.0, device="cpu")
    assert m == 1.0 and abs(turns[0].item() / 2.0**64 - 1 / (2 * math.pi)) < 1e-15


def test_binding_refuses_append_and_read(lib):
    x, slots = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int64)
    turns, _ = rq.rope_turns(64, device="cpu")
    bad = _cache()
    bad["ks"] = bad["ks"].double()
    for kw, match in [
        (dict(v=torch.zeros(3, 1, 64)), "v: expected shape"),
        (dict(cache=_cache(D=32)), "cache\\['kq'\\]: expected"),
        (dict(cache=_cache(H=3)), "cache holds 3 heads"),
        (dict(cache=bad), "scales float32"),
        (dict(slots=slots.int()), "slots must be"),
        (dict(positions=slots), "go together"),
        (dict(positions=slots[:1], turns=turns), "positions must be"),
        (dict(), "CUDA"),
    ]:
        args = dict(v=x, cache=_cache(), slots=slots, positions=None, turns=None) | kw
        with pytest.raises(ValueError, match=match):
            rq.kv_append(x, args["v"], args["cache"], args["slots"], 1, positions=args["positions"], turns=args["turns"])
    table, off = torch.zeros(1, 2, dtype=torch.int32), _i32(0, 5)
    for kw, match in [
        (dict(table=table[0]), "block_table must be"),
        (dict(table=table.long()), "block_table must be"),
        (dict(off=_i32(0, 2, 5)), "offsets must be"),
        (dict(starts=_i32(0, 0)), "starts must be"),
        (dict(dtype=torch.float64), "dtype must be"),
        (dict(out=(torch.zeros(5, 2, 64), torch.zeros(4, 2, 64))), "out \\(v\\): expected shape"),
        (dict(), "CUDA"),
    ]:
        args = dict(table=table, off=off, starts=None, dtype=torch.float32, out=None) | kw
        with pytest.raises(ValueError, match=match):
            rq.kv_read(_cache(), args["table"], args["starts"], args["off"], 5, 1, dtype=args["dtype"], out=args["out"])


def test_binding_refuses_attn_tree(lib):
    q, table = torch.zeros(3, 4, 64), torch.zeros(1, 2, dtype=torch.int32)
    for kw, match in [
        (dict(q=torch.zeros(3, 5, 64)), "do not divide"),
        (dict(q=q.double()), "float32, bfloat16 or float16"),
        (dict(table=table.long()), "block_table must be"),
        (dict(ctx=_i32(1, 2)), "context_lens must be"),
        (dict(off=_i32(0)), "offsets must be"),
        (dict(tree_mask=torch.ones(3, 3)), "tree_mask must be bool"),
        (dict(tree_mask=torch.ones(2, 3, dtype=torch.bool)), "tree_mask must be bool"),
        (dict(tree_mask=torch.ones(3, 3, dtype=torch.bool), max_nodes=4), "narrower than max_nodes"),
        (dict(out=torch.zeros(3, 4, 64, dtype=torch.bfloat16)), "out: expected dtype"),
        (dict(), "CUDA"),
    ]:
        args = dict(q=q, table=table, ctx=_i32(4), off=_i32(0, 3), tree_mask=None, max_nodes=None, out=None) | kw
        with pytest.raises(ValueError, match=match):
            rq.attn_tree(args["q"], _cache(), args["table"], args["ctx"], args["off"], 1, tree_mask=args["tree_mask"],
                         max_nodes=args["max_nodes"], out=args["out"])
