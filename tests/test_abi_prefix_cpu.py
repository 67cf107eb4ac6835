"""Host-side checks of the planning, shared-prefix and W4A16 entry points: bad arguments are refused before
anything is enqueued (these calls never touch a GPU).  And the plain forms that the GPU tests compare with."""
import ctypes

import pytest
import torch

import paged_ref
import prefix_ref
import rotational_w4a4_quantization_gb300 as rq
from rotational_w4a4_quantization_gb300 import build as rq_build

A16, A8, A4, A2, B16 = (ctypes.c_void_p(x) for x in (0x10000, 0x10008, 0x10004, 0x10002, 0x20000))
NULL = None


@pytest.fixture(scope="module")
def lib():
    rq_build.build()
    return rq.load_library()


def plan(lib, ctx=A16, new=A16, base=NULL, B=4, table=A16, W=3, free=A16, F=10, head=NULL, page=64, total=8, off=A16, slots=A16,
         pos=A16, after=B16):
    return lib.rq_kv_plan(ctx, new, base, B, table, W, free, F, head, page, total, off, slots, pos, after, NULL)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), 1),
    (dict(W=-1), 1),
    (dict(F=-1), 1),
    (dict(total=-1), 1),
    (dict(page=0), 1),
    (dict(page=24), 2),
    (dict(page=8), 2),
    (dict(page=512), 2),
    (dict(B=65537), 2),
    (dict(total=1 << 31), 2),
    (dict(W=1 << 26), 2),
    (dict(ctx=NULL), 1),
    (dict(new=NULL), 1),
    (dict(table=NULL), 1),
    (dict(free=NULL), 1),
    (dict(off=NULL), 1),
    (dict(slots=NULL), 1),
    (dict(pos=NULL), 1),
    (dict(after=NULL), 1),
    (dict(head=B16), 1),                # the step's own head
    (dict(ctx=A2), 3),
    (dict(base=A2), 3),
    (dict(head=A2), 3),
    (dict(slots=A4), 3),
    (dict(pos=A4), 3),
])
def test_plan_argument_checks(lib, kw, expect):
    assert plan(lib, **kw) == expect


def prefix(lib, q=A16, qt=4096, dt=1, N=8, Hq=32, D=128, kq=A16, pages=4, H=8, page=64, table=A16, W=2, ctx=A16, off=A16,
           B=2, ptable=A16, PW=2, lens=A16, groups=A16, G=1, nodes=4, mask=NULL, ms=0, flags=1, out=A16, ws=A16, wb=1 << 40):
    return lib.rq_attn_prefix(q, qt, 128, dt, N, Hq, D, kq, A16, A16, A16, pages, H, page, table, W, ctx, off, B, ptable, PW,
                              lens, groups, G, nodes, mask, ms, 7, flags, 0.088, out, ws, wb, NULL)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), 1),
    (dict(Hq=0), 1),
    (dict(B=-1), 1),
    (dict(G=-1), 1),
    (dict(PW=-1), 1),
    (dict(flags=4), 1),
    (dict(dt=3), 2),
    (dict(D=96), 2),
    (dict(page=8), 2),
    (dict(Hq=30), 1),
    (dict(mask=A16, ms=3), 1),
    (dict(pages=1 << 24), 2),
    (dict(PW=1 << 26), 2),
    (dict(N=1 << 26), 2),               # rows x heads past 2^30
    (dict(q=NULL), 1),
    (dict(table=NULL), 1),
    (dict(ptable=NULL), 1),
    (dict(PW=0), 1),
    (dict(lens=NULL), 1),
    (dict(groups=NULL), 1),
    (dict(ws=NULL), 1),
    (dict(wb=8 * 32 * 130 * 4 - 1), 1),  # less than the state alone
    (dict(q=A8), 3),
    (dict(ptable=A2), 3),
    (dict(lens=A2), 3),
    (dict(groups=A2), 3),
    (dict(N=0, q=NULL), 0),
    (dict(B=0, q=NULL), 0),
    (dict(nodes=0, q=NULL), 0),
])
def test_prefix_argument_checks(lib, kw, expect):
    assert prefix(lib, **kw) == expect


def w4a16(lib, x=A16, dt=1, M=4, K=256, ld=256, w=A16, s=A16, N=7, group=128, y=A16, yt=1):
    return lib.rq_w4a16_gemm(x, dt, M, K, ld, w, s, N, group, y, yt, NULL)


@pytest.mark.parametrize("kw,expect", [
    (dict(M=-1), 1),
    (dict(N=-1), 1),
    (dict(K=0), 1),
    (dict(group=0), 1),
    (dict(ld=255), 1),
    (dict(dt=3), 2),
    (dict(yt=3), 2),
    (dict(K=192), 2),
    (dict(group=64), 2),
    (dict(M=65), 2),
    (dict(K=262272, ld=262272), 2),
    (dict(N=1 << 31), 2),
    (dict(x=NULL), 1),
    (dict(w=NULL), 1),
    (dict(s=NULL), 1),
    (dict(y=NULL), 1),
    (dict(x=A8), 3),
    (dict(w=A8), 3),
    (dict(y=A8), 3),
    (dict(s=A2), 3),
    (dict(ld=260), 3),                  # 520-byte rows
    (dict(M=0, x=NULL), 0),
    (dict(N=0, w=NULL), 0),
])
def test_w4a16_argument_checks(lib, kw, expect):
    assert w4a16(lib, **kw) == expect


# ---- the binding, on CPU tensors: checks come before the device check ----

def _i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def test_binding_refuses_plan(lib):
    table = torch.zeros(2, 3, dtype=torch.int32)
    out = (_i32(0, 0, 0), torch.zeros(5, dtype=torch.int64), torch.zeros(5, dtype=torch.int64), _i32(0))
    for kw, match in [
        (dict(table=table.long()), "block_table must be"),
        (dict(table=table.t()), "block_table must be"),
        (dict(ctx=_i32(1)), "context_lens must be"),
        (dict(new=torch.ones(2)), "new_lens must be"),
        (dict(free=torch.zeros(4)), "free_pages must be"),
        (dict(free=torch.zeros(8, dtype=torch.int32)[::2]), "free_pages must be"),
        (dict(), "CUDA"),
    ]:
        a = dict(ctx=_i32(1, 2), new=_i32(1, 1), table=table, free=_i32(0, 1), head=None, base=None, out=None) | kw
        with pytest.raises(ValueError, match=match):
            rq.kv_plan(a["ctx"], a["new"], a["table"], a["free"], 5, 16, head=a["head"], base=a["base"], out=a["out"])
    assert out


def test_binding_refuses_prefix(lib):
    q, table, cache = torch.zeros(3, 4, 64), torch.zeros(1, 2, dtype=torch.int32), rq.kv_cache(2, 2, 64, 16, device="cpu")
    for kw, match in [
        (dict(q=torch.zeros(3, 5, 64)), "do not divide"),
        (dict(table=table.long()), "block_table must be"),
        (dict(tree_mask=torch.ones(3, 3)), "tree_mask must be bool"),
        (dict(), "CUDA"),
    ]:
        a = dict(q=q, table=table, tree_mask=None) | kw
        with pytest.raises(ValueError, match=match):
            rq.attn_prefix(a["q"], cache, a["table"], _i32(4), _i32(0, 3), table, _i32(9), _i32(0, 1), 1, tree_mask=a["tree_mask"])


def test_binding_refuses_w4a16(lib):
    x, w = torch.zeros(3, 256), torch.zeros(5, 128, dtype=torch.uint8)
    s = torch.ones(5, 2)
    for kw, match in [
        (dict(x=x[0]), "x must be 2-D"),
        (dict(x=torch.zeros(256, 3).t()), "x must be 2-D"),
        (dict(x=x.double()), "x must be float32"),
        (dict(w=w.to(torch.int8)), "w_q must be"),
        (dict(w=w[:, :64]), "w_q must be"),
        (dict(s=torch.ones(5, 3)), "w_scales must be"),
        (dict(s=torch.ones(4)), "w_scales must be"),
        (dict(s=s.double()), "w_scales must be"),
        (dict(out_dtype=torch.int32), "out_dtype must be"),
        (dict(out=torch.zeros(3, 4)), "out: expected shape"),
        (dict(out=torch.zeros(3, 5, dtype=torch.int32)), "out: expected dtype"),
        (dict(), "CUDA"),
    ]:
        a = dict(x=x, w=w, s=s, out=None, out_dtype=None) | kw
        with pytest.raises(ValueError, match=match):
            rq.w4a16_gemm(a["x"], a["w"], a["s"], out=a["out"], out_dtype=a["out_dtype"])


# ---- the plain forms ----

def test_plan_by_hand():
    """Two requests, pages of 4: the first has 5 tokens on pages 7, 8 and gets 4; the second is new and gets 5."""
    offsets, slots, positions, head, table = prefix_ref.plan([5, 0], [4, 5], [[7, 8, 3], [9, 9, 9]], [1, 0, 2, 5], 10, 4, head=1,
                                                             base=[100, 0])
    assert offsets == [0, 4, 9] and head == 4 and table == [[7, 8, 0], [2, 5, -1]]
    assert slots == [33, 34, 35, 0, 8, 9, 10, 11, 20, -1]
    assert positions == [105, 106, 107, 108, 0, 1, 2, 3, 4, 0]


def test_joined_tables_name_prefix_and_own_tokens():
    page = 4
    cache = {n: torch.arange(6 * 2 * page).view(6, 2, page, *([1] if n[1] == "q" else [])) for n in ("kq", "ks", "vq", "vs")}
    flat, table, ctx = prefix_ref.joined(cache, torch.tensor([[3, 0], [9, 1]]), [2, 0], [3, 1], torch.tensor([[5]]),
                                         [3], torch.tensor([1, 2]))
    assert ctx.tolist() == [2, 3]
    assert table.tolist() == [[12, 13, 14, 15, 0], [20, 21, 22, -1, -1]]       # page 9 is not there
    assert flat["ks"][21, :, 0].tolist() == cache["ks"][5, :, 1].tolist()


def test_weights_of_the_plain_form():
    codes = torch.tensor([[0x1F, 0x80]], dtype=torch.uint8)
    assert prefix_ref.weights(codes, torch.tensor([2.0])).tolist() == [[-2.0, 2.0, 0.0, -16.0]]
    assert paged_ref.UNIT[torch.float16] == 2.0**-11
