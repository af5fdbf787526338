"""Refusals of the scored router, of the product with an MXFP4 matrix and of the
experts' combine: the C entries' checks (no GPU is touched) and the binding's."""
import os
import warnings

import pytest
import torch

import mxfp4_routed_expert_topk_amd as moe

BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        pytest.fail(f"library not built at {moe.LIB_PATH}: run python -m mxfp4_routed_expert_topk_amd.build")
    return moe.load_library()


def refused(lib, fn, args, status, needle):
    assert getattr(lib, fn)(*args) == status, (fn, args)
    assert needle in lib.moe_mxfp4_last_error().decode(), lib.moe_mxfp4_last_error()


P = 4096   # a pointer that is aligned and never read

SELECT = dict(logits=P, dtype=1, ldl=24, T=4, E=24, k=3, score=0, bias=None, groups=4, limit=2, top=1, renorm=1, scale=1.0,
              ids=P, weights=P, stream=None)


@pytest.mark.parametrize("change,status,needle", [
    (dict(dtype=2), 1, "dtype must be"),
    (dict(T=-1), 1, "num_tokens must be >= 0"),
    (dict(T=(1 << 24) + 1), 2, "num_tokens must be at most"),
    (dict(E=0), 2, "num_experts must be in [1, 1024]"),
    (dict(E=1025, ldl=1025), 2, "num_experts must be in [1, 1024]"),
    (dict(k=0), 2, "top_k must be in [1, min(32, num_experts=24)]"),
    (dict(k=25), 2, "top_k must be in"),
    (dict(E=64, ldl=64, k=33, limit=4), 2, "top_k must be in"),
    (dict(score=2), 1, "score must be"),
    (dict(score=-1), 1, "score must be"),
    (dict(scale=NAN), 1, "scale must be finite"),
    (dict(scale=INF), 1, "scale must be finite"),
    (dict(ldl=23), 2, "ldl must be"),
    (dict(ldl=(1 << 20) + 1), 2, "ldl must be"),
    (dict(groups=0), 2, "num_groups must divide num_experts=24"),
    (dict(groups=5), 2, "num_groups must divide num_experts=24"),
    (dict(E=128, ldl=128, groups=128), 2, "num_groups must divide"),
    (dict(limit=0), 2, "group_limit must be in [1, num_groups=4]"),
    (dict(limit=5), 2, "group_limit must be in"),
    (dict(top=0), 2, "group_top must be 1 or 2"),
    (dict(top=3), 2, "group_top must be 1 or 2"),
    (dict(k=13), 2, "top_k=13 is more than the 12 experts"),
    (dict(logits=None), 1, "logits is null"),
    (dict(logits=P + 2), 3, "logits must be 4-byte aligned"),
    (dict(dtype=0, logits=P + 1), 3, "logits must be 2-byte aligned"),
    (dict(bias=P + 2), 3, "bias must be 4-byte aligned"),
    (dict(ids=None), 1, "topk_ids is null"),
    (dict(weights=P + 2), 3, "topk_weights must be 4-byte aligned"),
])
def test_select_refusals(lib, change, status, needle):
    refused(lib, "moe_router_select", tuple({**SELECT, **change}.values()), status, needle)


SELECT_BACK = dict(dweights=P, logits=P, dtype=1, ldl=24, ids=P, T=4, E=24, k=3, score=0, renorm=1, scale=1.0, dlogits=P,
                   stream=None)


@pytest.mark.parametrize("change,status,needle", [
    (dict(dtype=5), 1, "dtype must be"),
    (dict(T=-2), 1, "num_tokens must be >= 0"),
    (dict(E=1025, ldl=1025), 2, "num_experts must be"),
    (dict(k=33, E=40, ldl=40), 2, "top_k must be"),
    (dict(ldl=3), 2, "ldl must be"),
    (dict(score=9), 1, "score must be"),
    (dict(scale=-INF), 1, "scale must be finite"),
    (dict(dweights=None), 1, "dweights is null"),
    (dict(ids=P + 1), 3, "topk_ids must be 4-byte aligned"),
    (dict(dlogits=P + 4), 3, "dlogits must be 16-byte aligned"),
])
def test_select_backward_refusals(lib, change, status, needle):
    refused(lib, "moe_router_select_backward", tuple({**SELECT_BACK, **change}.values()), status, needle)


LINEAR = dict(x=P, ldx=64, codes=P, scales=P, m=4, n=6, k=64, gate=0, dtype=0, out=P, stream=None)


@pytest.mark.parametrize("change,status,needle", [
    (dict(dtype=-1), 1, "dtype must be"),
    (dict(m=-1), 1, "m and n must be >= 0"),
    (dict(n=(1 << 19) + 2), 2, "m and n must be at most"),
    (dict(k=48), 2, "k must be a multiple of 32"),
    (dict(k=65568, ldx=65568), 2, "k must be a multiple of 32"),
    (dict(gate=1, n=7), 2, "a gated product needs an even n"),
    (dict(ldx=56), 2, "ldx must be"),
    (dict(ldx=68), 2, "ldx must be a multiple of 8"),
    (dict(x=P + 2), 3, "x must be 16-byte aligned"),
    (dict(codes=P + 8), 3, "codes must be 16-byte aligned"),
    (dict(scales=None), 1, "scales is null"),
    (dict(out=None), 1, "out is null"),
])
def test_linear_refusals(lib, change, status, needle):
    refused(lib, "moe_mxfp4_linear", tuple({**LINEAR, **change}.values()), status, needle)


COMBINE = dict(y=P, ldy=64, rows=12, rowpos=P, weights=P, T=4, k=3, H=64, dtype=0, out=P, stream=None)


@pytest.mark.parametrize("change,status,needle", [
    (dict(dtype=2), 1, "dtype must be"),
    (dict(rows=-1), 1, "rows and num_tokens must be >= 0"),
    (dict(T=-1), 1, "rows and num_tokens must be >= 0"),
    (dict(rows=(1 << 26) + 1), 2, "rows must be at most"),
    (dict(T=(1 << 21) + 1), 2, "num_tokens must be at most"),
    (dict(k=0), 2, "top_k must be in [1, 32]"),
    (dict(k=33), 2, "top_k must be in [1, 32]"),
    (dict(H=60), 2, "hidden must be a multiple of 8"),
    (dict(H=0), 2, "hidden must be a multiple of 8"),
    (dict(H=65544, ldy=65544), 2, "hidden must be a multiple of 8"),
    (dict(ldy=56), 2, "ldy must be"),
    (dict(ldy=68), 2, "ldy must be a multiple of 8"),
    (dict(y=None), 1, "y is null"),
    (dict(y=P + 8), 3, "y must be 16-byte aligned"),
    (dict(rowpos=P + 2), 3, "rowpos must be 4-byte aligned"),
    (dict(weights=P + 1), 3, "weights must be 4-byte aligned"),
    (dict(out=P + 4), 3, "out must be 16-byte aligned"),
])
def test_combine_refusals(lib, change, status, needle):
    refused(lib, "moe_expert_combine", tuple({**COMBINE, **change}.values()), status, needle)


COMBINE_BACK = dict(dout=P, dtype=0, lddout=64, y=P, ldy=64, rows=12, rowpos=P, perm=P, weights=P, T=4, k=3, H=64, dy=P,
                    dweights=P, stream=None)


@pytest.mark.parametrize("change,status,needle", [
    (dict(dtype=7), 1, "dout_dtype must be"),
    (dict(lddout=72 + 4), 2, "lddout must be a multiple of 8"),
    (dict(dtype=1, lddout=70), 2, "lddout must be a multiple of 4"),
    (dict(lddout=56), 2, "lddout must be"),
    (dict(ldy=0), 2, "ldy must be"),
    (dict(H=12), 2, "hidden must be a multiple of 8"),
    (dict(rows=-5), 1, "rows and num_tokens must be >= 0"),
    (dict(dout=None), 1, "dout is null"),
    (dict(perm=None), 1, "perm is null"),
    (dict(y=None), 1, "y is null"),
    (dict(rowpos=None), 1, "rowpos is null"),
    (dict(dy=P + 8), 3, "dy must be 16-byte aligned"),
    (dict(dweights=P + 2), 3, "dweights must be 4-byte aligned"),
])
def test_combine_backward_refusals(lib, change, status, needle):
    refused(lib, "moe_expert_combine_backward", tuple({**COMBINE_BACK, **change}.values()), status, needle)


def test_empty_calls_are_no_ops(lib):
    none = lambda base, **change: tuple({**{k: None if v == P else v for k, v in base.items()}, **change}.values())
    assert lib.moe_router_select(*none(SELECT, T=0)) == 0
    assert lib.moe_router_select_backward(*none(SELECT_BACK, T=0)) == 0
    assert lib.moe_mxfp4_linear(*none(LINEAR, m=0)) == 0
    assert lib.moe_mxfp4_linear(*none(LINEAR, n=0, gate=1)) == 0
    assert lib.moe_expert_combine(*none(COMBINE, T=0)) == 0
    assert lib.moe_expert_combine_backward(*none(COMBINE_BACK, T=0)) == 0
    assert lib.moe_expert_combine_backward(*none(COMBINE_BACK)) == 0                       # no gradient wanted
    assert lib.moe_expert_combine_backward(*none(COMBINE_BACK, rows=0, dy=P, ldy=0)) == 0  # no rows to write


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def f(*shape):
    return z(*shape, dtype=F32)


def i(*shape):
    return z(*shape, dtype=I32)


def u(*shape):
    return z(*shape, dtype=U8)


@pytest.mark.parametrize("call,status,needle", [
    (lambda: moe.router_select([1.0], 1), 1, "logits must be a torch.Tensor"),
    (lambda: moe.router_select(z(4, 8, dtype=torch.float16), 1), 1, "logits must be torch.float32 or torch.bfloat16"),
    (lambda: moe.router_select(f(8), 1), 1, "logits must be [rows, cols]"),
    (lambda: moe.router_select(f(8, 8).t(), 1), 1, "rows of logits must be contiguous"),
    (lambda: moe.router_select(f(4, 8), 9), 2, "top_k must be in [1, 8]"),
    (lambda: moe.router_select(f(4, 8), -1), 2, "top_k must be in [1, 8]"),
    (lambda: moe.router_select(f(4, 8), 2, bias=f(7)), 1, "bias must have shape (8,)"),
    (lambda: moe.router_select(f(4, 8), 2, bias=z(8)), 1, "bias must be torch.float32"),
    (lambda: moe.router_select(f(4, 8), 2, ids=i(4, 3)), 1, "ids must have shape (4, 2)"),
    (lambda: moe.router_select(f(4, 8), 2, weights=z(4, 2)), 1, "weights must be torch.float32"),
    (lambda: moe.router_select(f(4, 8), 2, num_groups=(1 << 32) + 1), 2, "must be below 2^31"),
    (lambda: moe.router_select(f(4, 8), 2), 1, "must be on a GPU"),
    (lambda: moe.router_select_backward(f(4, 2), f(4, 8), None), 1, "ids must be a 2-D"),
    (lambda: moe.router_select_backward(f(4, 2), f(4, 8), i(3, 2)), 1, "ids must have shape (4, 2)"),
    (lambda: moe.router_select_backward(f(4, 3), f(4, 8), i(4, 2)), 1, "dweights must have shape (4, 2)"),
    (lambda: moe.router_select_backward(f(4, 2), z(4, 8), i(4, 2), dlogits=f(4, 8)), 1, "dlogits must be torch.bfloat16"),
    (lambda: moe.router_select_backward(f(4, 2), f(4, 8), i(4, 2)), 1, "must be on a GPU"),
    (lambda: moe.mxfp4_linear(z(4, 32), u(5, 32), u(5, 2)), 1, "x must be [rows, 64]"),
    (lambda: moe.mxfp4_linear(f(4, 64), u(5, 32), u(5, 2)), 1, "x must be torch.bfloat16"),
    (lambda: moe.mxfp4_linear(z(4, 64), u(5, 32), u(5, 3)), 1, "scales must have shape (5, 2)"),
    (lambda: moe.mxfp4_linear(z(4, 64), u(5, 32), u(5, 2), gate=True), 2, "needs an even n, got 5"),
    (lambda: moe.mxfp4_linear(z(4, 64), u(6, 32), u(6, 2), gate=True, out=z(4, 6)), 1, "out must have shape (4, 3)"),
    (lambda: moe.mxfp4_linear(z(4, 64), u(6, 32), u(6, 2), dtype=torch.float16), 1, "dtype must be"),
    (lambda: moe.mxfp4_linear(z(4, 64), u(6, 32), u(6, 2)), 1, "must be on a GPU"),
    (lambda: moe.expert_combine(f(8, 16), i(4, 2)), 1, "y must be torch.bfloat16"),
    (lambda: moe.expert_combine(z(8, 16), i(8)), 1, "rowpos must be a 2-D"),
    (lambda: moe.expert_combine(z(8, 16), z(4, 2, dtype=torch.int64)), 1, "rowpos must be torch.int32"),
    (lambda: moe.expert_combine(z(8, 16), i(4, 2), f(4, 3)), 1, "weights must have shape (4, 2)"),
    (lambda: moe.expert_combine(z(8, 16), i(4, 2), out=z(8, 16)), 1, "out must have shape (4, 16)"),
    (lambda: moe.expert_combine(z(8, 16), i(4, 2)), 1, "must be on a GPU"),
    (lambda: moe.expert_combine_backward(z(4, 16), z(8, 16), i(3, 2), i(8)), 1, "dout must have rowpos's 3 rows"),
    (lambda: moe.expert_combine_backward(z(4, 16), z(8, 24), i(4, 2), i(8)), 1, "y must be [rows, 16]"),
    (lambda: moe.expert_combine_backward(z(4, 16), z(8, 16), i(4, 2), i(7)), 1, "perm must have shape (8,)"),
    (lambda: moe.expert_combine_backward(z(4, 16), z(8, 16), i(4, 2)), 1, "perm must be a torch.Tensor"),
    (lambda: moe.expert_combine_backward(z(4, 16), None, i(4, 2), None, need_dw=False), 1, "perm must be a 1-D"),
    (lambda: moe.expert_combine_backward(z(4, 16), None, i(4, 2), i(8)), 1, "y must be a torch.Tensor"),
    (lambda: moe.expert_combine_backward(z(4, 16), z(8, 16), i(4, 2), i(8), dy=z(4, 16)), 1, "dy must have shape (8, 16)"),
    (lambda: moe.expert_combine_backward(z(4, 16), z(8, 16), i(4, 2), dy=z(8, 16), need_dy=False), 1,
     "dy is given, but need_dy is False"),
    (lambda: moe.expert_combine_backward(z(4, 16), None, i(4, 2), i(8), dweights=f(4, 2), need_dw=False), 1,
     "dweights is given, but need_dw is False"),
    (lambda: moe.expert_combine_backward(z(4, 16), None, i(4, 2), need_dy=False, need_dw=False), 1,
     "need_dy or need_dw must be True"),
    (lambda: moe.expert_combine_backward(z(4, 16), z(8, 16), i(4, 2), i(8)), 1, "must be on a GPU"),
])
def test_binding_refusals(lib, call, status, needle):
    with pytest.raises(moe.MoeError) as ei:
        call()
    assert ei.value.status == status and needle in ei.value.message, ei.value.message


def test_binding_refuses_overlapping_outputs(lib):
    both = f(4, 8)
    with pytest.raises(moe.MoeError, match="weights must not overlap logits"):
        moe.router_select(both, 8, weights=both)
    ids = i(4, 2)
    with pytest.raises(moe.MoeError, match="weights must not overlap ids"):
        moe.router_select(f(4, 8), 2, ids=ids, weights=ids.view(F32))
    with pytest.raises(moe.MoeError, match="dlogits must not overlap logits"):
        moe.router_select_backward(f(4, 2), both, i(4, 2), dlogits=both)
    x = z(8, 64)
    with pytest.raises(moe.MoeError, match="out must not overlap x"):
        moe.mxfp4_linear(x, u(64, 32), u(64, 2), out=x)
    with pytest.raises(moe.MoeError, match="out must not overlap y"):
        moe.expert_combine(x, i(8, 1), out=x)
    with pytest.raises(moe.MoeError, match="dy must not overlap y"):
        moe.expert_combine_backward(z(4, 64), x, i(4, 2), i(8), dy=x)
    with pytest.raises(moe.MoeError, match="dweights must not overlap weights"):
        w = f(4, 2)
        moe.expert_combine_backward(z(4, 64), x, i(4, 2), i(8), w, dweights=w)


BIG = 1 << 32                       # sizes reach the C entries as int32, where BIG + n would count as n


def m(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("call,needle", [
    (lambda: moe.router_select(m(BIG + 1, 8, dtype=F32), 2), f"num_tokens={BIG + 1}"),
    (lambda: moe.router_select(m(1, BIG + 8), 2), f"num_experts={BIG + 8}"),
    (lambda: moe.router_select(m(4, 8), 2, group_limit=BIG + 1), f"group_limit={BIG + 1}"),
    (lambda: moe.router_select_backward(m(BIG, 2, dtype=F32), m(BIG, 8), m(BIG, 2, dtype=I32)), f"num_tokens={BIG}"),
    (lambda: moe.router_select_backward(m(1, BIG + 2, dtype=F32), m(1, 8), m(1, BIG + 2, dtype=I32)), f"top_k={BIG + 2}"),
    (lambda: moe.mxfp4_linear(m(BIG + 1, 32), m(2, 16, dtype=U8), m(2, 1, dtype=U8)), f"m={BIG + 1}"),
    (lambda: moe.mxfp4_linear(m(1, 32), m(BIG + 2, 16, dtype=U8), m(BIG + 2, 1, dtype=U8)), f"rows={BIG + 2}"),
    (lambda: moe.expert_combine(m(BIG + 8, 8), m(1, 1, dtype=I32)), f"rows={BIG + 8}"),
    (lambda: moe.expert_combine(m(8, BIG + 8), m(1, 1, dtype=I32)), f"hidden={BIG + 8}"),
    (lambda: moe.expert_combine(m(8, 8), m(BIG + 1, 1, dtype=I32)), f"num_tokens={BIG + 1}"),
    (lambda: moe.expert_combine_backward(m(2, 8), m(BIG + 8, 8), m(2, 1, dtype=I32), m(BIG + 8, dtype=I32)),
     f"rows={BIG + 8}"),
])
def test_sizes_that_no_int32_holds_are_refused(lib, call, needle):
    with pytest.raises(moe.MoeError) as ei:
        call()
    assert ei.value.status == 2 and needle in ei.value.message, ei.value.message


@pytest.mark.parametrize("change,status,needle", [
    (dict(num_groups=2 - BIG), 2, f"num_groups={2 - BIG}"),
    (dict(num_groups=4, group_limit=2 - BIG), 2, f"group_limit={2 - BIG}"),
    (dict(group_top=1 - BIG), 2, f"group_top={1 - BIG}"),
    (dict(top_k=2 - BIG), 2, "top_k"),
    (dict(num_groups=-1, group_top=BIG + 1), 2, f"group_top={BIG + 1}"),   # a negative one does not hide a large one
    (dict(num_groups=-4), 2, "num_groups must divide num_experts=8 and be in [1, 64], got -4"),
    (dict(num_groups=-2 ** 31), 2, "num_groups must divide"),
    (dict(group_limit=-1), 2, "group_limit must be in"),
    (dict(group_top=-1), 2, "group_top must be 1 or 2"),
    (dict(score=BIG), 1, f"got {BIG}"),                                   # its low 32 bits are softmax's
    (dict(score=1 - BIG), 1, "score must be"),
    (dict(score=2), 1, "score must be MOE_SCORE_SOFTMAX (0) or MOE_SCORE_SIGMOID (1), got 2"),
    (dict(score="sigmoid"), 1, "score must be"),
    (dict(score=None), 1, "score must be"),
])
def test_select_refuses_what_no_int32_holds(lib, monkeypatch, change, status, needle):
    """Arguments reach the C entry as int32; what it refuses it refuses on the values given."""
    def launch(fn, args, like, stream, tensors):
        moe._check(fn(*args, None))
    monkeypatch.setattr(moe, "_launch", launch)   # tensors of no rows: nothing is enqueued
    kw = {"top_k": 2, **change}
    with pytest.raises(moe.MoeError) as ei:
        moe.router_select(f(0, 8), **kw)
    assert ei.value.status == status and needle in ei.value.message, ei.value.message
    if "score" in change:
        with pytest.raises(moe.MoeError) as ei:
            moe.router_select_backward(f(0, 2), f(0, 8), i(0, 2), **change)
        assert ei.value.status == status and needle in ei.value.message, ei.value.message


@pytest.mark.parametrize("call,name", [
    (lambda t: moe.router_select(t["logits"], 2), "logits"),
    (lambda t: moe.mxfp4_linear(t["x"], u(4, 32), u(4, 2)), "x"),
    (lambda t: moe.expert_combine(t["x"], i(4, 2), t["w"]), "x"),
    (lambda t: moe.expert_combine(t["x"], i(4, 2), t["w"]), "w"),
])
def test_a_gradient_that_would_be_lost_is_warned_of(lib, call, name):
    t = {"logits": f(4, 8), "x": z(4, 64), "w": f(4, 2)}
    t[name].requires_grad_()

    def run():
        with pytest.raises(moe.MoeError, match="must be on a GPU"):
            call(t)

    with pytest.warns(UserWarning, match="records no autograd graph") as seen:
        run()
    assert seen[0].filename == __file__
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with torch.no_grad():
            run()
        t[name].requires_grad_(False)
        run()
