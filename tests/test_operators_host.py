"""Refusals of the MXFP4 quantiser and product and of the grouped products:
the C entries' checks (no GPU is touched) and the binding's."""
import os
import warnings

import pytest
import torch

import mxfp4_routed_expert_topk_amd as moe

BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        pytest.fail(f"library not built at {moe.LIB_PATH}: run python -m mxfp4_routed_expert_topk_amd.build")
    return moe.load_library()


def refused(lib, fn, args, status, needle):
    assert getattr(lib, fn)(*args) == status, (fn, args)
    assert needle in lib.moe_mxfp4_last_error().decode(), lib.moe_mxfp4_last_error()


P = 64   # a pointer that is aligned and never read


@pytest.mark.parametrize("args,status,needle", [
    ((P, 2, 4, 64, 64, P, P, None), 1, "dtype must be MOE_BF16"),
    ((P, 0, -1, 64, 64, P, P, None), 1, "rows must be >= 0"),
    ((P, 0, (1 << 24) + 1, 64, 64, P, P, None), 2, "rows must be at most"),
    ((P, 0, 4, 48, 48, P, P, None), 2, "multiple of 32"),
    ((P, 0, 4, 0, 0, P, P, None), 2, "multiple of 32"),
    ((P, 0, 4, 64, 32, P, P, None), 2, "ldx must be"),
    ((P, 0, 4, 64, 68, P, P, None), 2, "ldx must be a multiple of 8"),
    ((P, 1, 4, 64, 66, P, P, None), 2, "ldx must be a multiple of 4"),
    ((None, 0, 4, 64, 64, P, P, None), 1, "x is null"),
    ((P, 0, 4, 64, 64, P + 4, P, None), 3, "codes must be 16-byte aligned"),
    ((P, 0, 4, 64, 64, P, None, None), 1, "scales is null"),
    ((P + 8, 0, 4, 64, 64, P, P + 1, None), 3, "x must be 16-byte aligned"),
])
def test_quantize_refusals(lib, args, status, needle):
    refused(lib, "moe_mxfp4_quantize", args, status, needle)


@pytest.mark.parametrize("args,status,needle", [
    ((P, P, 4, 64, 3, P, None), 1, "dtype must be"),
    ((P, P, -4, 64, 0, P, None), 1, "rows must be >= 0"),
    ((P, P, 4, 33, 0, P, None), 2, "multiple of 32"),
    ((P, None, 4, 64, 0, P, None), 1, "scales is null"),
    ((P, P, 4, 64, 1, P + 8, None), 3, "out must be 16-byte aligned"),
])
def test_dequantize_refusals(lib, args, status, needle):
    refused(lib, "moe_mxfp4_dequantize", args, status, needle)


@pytest.mark.parametrize("args,status,needle", [
    ((P, P, P, P, 4, 4, 64, -1, P, None), 1, "dtype must be"),
    ((P, P, P, P, -1, 4, 64, 0, P, None), 1, "m and n must be >= 0"),
    ((P, P, P, P, 4, (1 << 19) + 1, 64, 0, P, None), 2, "m and n must be at most"),
    ((P, P, P, P, 4, 4, 40, 0, P, None), 2, "k must be a multiple of 32"),
    ((P, P, P, P, 4, 4, 0, 0, P, None), 2, "k must be a multiple of 32"),
    ((P, P, P, P, 4, 4, 65568, 0, P, None), 2, "k must be a multiple of 32"),
    ((P, P, None, P, 4, 4, 64, 0, P, None), 1, "b_codes is null"),
    ((P, P + 1, P + 2, P, 4, 4, 64, 0, P, None), 3, "b_codes must be 16-byte aligned"),
])
def test_matmul_refusals(lib, args, status, needle):
    refused(lib, "moe_mxfp4_matmul", args, status, needle)


@pytest.mark.parametrize("args,status,needle", [
    ((P, 64, P, P, -1, 2, 16, 64, P, None, 0, None), 1, "rows must be >= 0"),
    ((P, 64, P, P, (1 << 24) + 1, 2, 16, 64, P, None, 0, None), 2, "rows must be at most"),
    ((P, 64, P, P, 4, -1, 16, 64, P, None, 0, None), 1, "num_groups must be >= 0"),
    ((P, 64, P, P, 4, 4097, 16, 64, P, None, 0, None), 2, "num_groups must be at most"),
    ((P, 64, P, P, 4, 2, 12, 64, P, None, 0, None), 2, "n must be a multiple of 8"),
    ((P, 64, P, P, 4, 2, 0, 64, P, None, 0, None), 2, "n must be a multiple of 8"),
    ((P, 65, P, P, 4, 2, 16, 65, P, None, 0, None), 2, "k must be a multiple of 8"),
    ((P, 65544, P, P, 4, 2, 16, 65544, P, None, 0, None), 2, "k must be a multiple of 8"),
    ((P, 56, P, P, 4, 2, 16, 64, P, None, 0, None), 2, "ldx must be"),
    ((P, 68, P, P, 4, 2, 16, 64, P, None, 0, None), 2, "ldx must be a multiple of 8"),
    ((P, (1 << 20) + 8, P, P, 4, 2, 16, 64, P, None, 0, None), 2, "ldx must be"),
    ((P, 64, None, P, 4, 2, 16, 64, P, None, 0, None), 1, "w is null"),
    ((P, 64, P, P + 2, 4, 2, 16, 64, P, None, 0, None), 3, "offsets must be 4-byte aligned"),
])
def test_grouped_matmul_refusals(lib, args, status, needle):
    refused(lib, "moe_grouped_matmul", args, status, needle)


@pytest.mark.parametrize("args,status,needle", [
    ((P, 16, P, 64, P, P, 4, 2, 16, 64, P, P, 7, None, 0, None), 1, "dw_dtype must be"),
    ((P, 8, P, 64, P, P, 4, 2, 16, 64, P, P, 0, None, 0, None), 2, "lddy must be"),
    ((P, 16, P, 56, P, P, 4, 2, 16, 64, P, P, 0, None, 0, None), 2, "ldx must be"),
    ((P, 16, P, 64, P, P, -4, 2, 16, 64, P, P, 0, None, 0, None), 1, "rows must be >= 0"),
    ((P, 16, P, 64, P, P, 4, 2, 20, 64, P, P, 0, None, 0, None), 2, "n must be a multiple of 8"),
    ((None, 16, P, 64, P, P, 4, 2, 16, 64, P, P, 0, None, 0, None), 1, "dy is null"),
    ((P, 16, None, 64, P, P, 4, 2, 16, 64, None, P, 0, None, 0, None), 1, "x is null"),
    ((P, 16, P, 64, None, P, 4, 2, 16, 64, P, None, 0, None, 0, None), 1, "w is null"),
    ((P, 16, P, 64, P, None, 4, 2, 16, 64, P, P, 0, None, 0, None), 1, "offsets is null"),
    ((P, 16, P, 64, P, P, 4, 2, 16, 64, P + 8, None, 0, None, 0, None), 3, "dx must be 16-byte aligned"),
    ((P, 16, P, 64, P, P, 4, 2, 16, 64, None, P + 2, 0, None, 0, None), 3, "dw must be 16-byte aligned"),
])
def test_grouped_backward_refusals(lib, args, status, needle):
    refused(lib, "moe_grouped_matmul_backward", args, status, needle)


def test_empty_calls_are_no_ops(lib):
    assert lib.moe_mxfp4_quantize(None, 0, 0, 64, 64, None, None, None) == 0
    assert lib.moe_mxfp4_dequantize(None, None, 0, 64, 0, None, None) == 0
    assert lib.moe_mxfp4_matmul(None, None, None, None, 0, 5, 64, 0, None, None) == 0
    assert lib.moe_mxfp4_matmul(None, None, None, None, 5, 0, 64, 0, None, None) == 0
    assert lib.moe_grouped_matmul(None, 64, None, None, 0, 2, 16, 64, None, None, 0, None) == 0
    assert lib.moe_grouped_matmul(None, 64, None, None, 4, 0, 16, 64, None, None, 0, None) == 0
    assert lib.moe_grouped_matmul_backward(None, 16, None, 64, None, None, 4, 0, 16, 64, None, None, 0, None, 0, None) == 0
    assert lib.moe_grouped_matmul_backward(None, 16, None, 64, None, None, 4, 2, 16, 64, None, None, 0, None, 0, None) == 0
    assert lib.moe_grouped_matmul_backward(None, 16, None, 64, None, None, 0, 2, 16, 64, P, None, 0, None, 0, None) == 0


def test_grouped_workspaces(lib):
    fwd, bwd = lib.moe_grouped_matmul_workspace, lib.moe_grouped_matmul_backward_workspace
    # many tiles, short sums, nothing to do, sizes that the entries refuse: none
    assert fwd(32768, 8, 4096, 7168) == fwd(32, 8, 256, 256) == fwd(0, 8, 64, 7168) == fwd(9, 0, 64, 7168) == 0
    assert fwd(9, 2, 63, 7168) == bwd(6566, 1, 584, 184, 0, 0) == bwd(12288, 32, 4096, 7168, 1, 1) == 0
    need = fwd(718, 1, 64, 6672)
    assert need > 0 and need % (718 * 64 * 4) == 0       # whole fp32 copies of y
    assert bwd(6566, 1, 584, 184, 0, 1) % (584 * 184 * 4) == 0 < bwd(6566, 1, 584, 184, 0, 1)
    refused(lib, "moe_grouped_matmul", (P, 6672, P, P, 718, 1, 64, 6672, P, P, need - 1, None), 4,
            f"workspace must hold {need} bytes")
    refused(lib, "moe_grouped_matmul", (P, 6672, P, P, 718, 1, 64, 6672, P, P + 8, need, None), 3,
            "workspace must be 16-byte aligned")
    refused(lib, "moe_grouped_matmul_backward",
            (P, 584, P, 184, P, P, 6566, 1, 584, 184, P, P, 0, P, 64, None), 4, "workspace must hold")


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("call,status,needle", [
    (lambda: moe.mxfp4_quantize([1.0]), 1, "x must be a torch.Tensor"),
    (lambda: moe.mxfp4_quantize(z(4, 64, dtype=torch.float16)), 1, "x must be torch.bfloat16 or torch.float32"),
    (lambda: moe.mxfp4_quantize(z(64)), 1, "x must be [rows, cols]"),
    (lambda: moe.mxfp4_quantize(z(4, 48)), 2, "multiple of 32"),
    (lambda: moe.mxfp4_quantize(z(4, 128)[:, ::2]), 1, "rows of x must be contiguous"),
    (lambda: moe.mxfp4_quantize(z(64, 64).t()), 1, "rows of x must be contiguous"),
    (lambda: moe.mxfp4_quantize(z(4, 64), codes=z(4, 64, dtype=U8)), 1, "codes must have shape (4, 32)"),
    (lambda: moe.mxfp4_quantize(z(4, 64), scales=z(4, 2)), 1, "scales must be torch.uint8"),
    (lambda: moe.mxfp4_quantize(z(4, 64)), 1, "must be on a GPU"),
    (lambda: moe.mxfp4_dequantize(z(4, 32), z(4, 2, dtype=U8)), 1, "codes must be torch.uint8"),
    (lambda: moe.mxfp4_dequantize(z(4, 24, dtype=U8), z(4, 1, dtype=U8)), 2, "positive multiple of 16 columns"),
    (lambda: moe.mxfp4_dequantize(z(4, 32, dtype=U8), z(4, 3, dtype=U8)), 1, "scales must have shape (4, 2)"),
    (lambda: moe.mxfp4_dequantize(z(4, 32, dtype=U8), z(4, 2, dtype=U8), dtype=torch.float16), 1, "dtype must be"),
    (lambda: moe.mxfp4_dequantize(z(4, 32, dtype=U8), z(4, 2, dtype=U8), dtype=BF, out=z(4, 64, dtype=F32)), 1,
     "out must be torch.bfloat16"),
    (lambda: moe.mxfp4_dequantize(z(4, 32, dtype=U8), z(4, 2, dtype=U8)), 1, "must be on a GPU"),
    (lambda: moe.mxfp4_matmul(z(4, 32, dtype=U8), z(4, 2, dtype=U8), z(5, 16, dtype=U8), z(5, 1, dtype=U8)), 2,
     "A has 64 columns and B 32"),
    (lambda: moe.mxfp4_matmul(z(4, 64, dtype=U8)[:, ::2], z(4, 2, dtype=U8), z(5, 32, dtype=U8), z(5, 2, dtype=U8)), 1,
     "a_codes must be contiguous"),
    (lambda: moe.mxfp4_matmul(z(4, 32, dtype=U8), z(4, 2, dtype=U8), z(5, 32, dtype=U8), z(5, 2, dtype=U8),
                              out=z(4, 4)), 1, "out must have shape (4, 5)"),
    (lambda: moe.grouped_matmul(z(4, 64), z(2, 16, 32), z(3, dtype=I32)), 1, "x must be [rows, 32]"),
    (lambda: moe.grouped_matmul(z(4, 64), z(2, 16, 64), z(3, dtype=torch.int64)), 1, "offsets must be torch.int32"),
    (lambda: moe.grouped_matmul(z(4, 64), z(2, 16, 64), z(2, dtype=I32)), 1, "offsets must have shape (3,)"),
    (lambda: moe.grouped_matmul(z(4, 64), z(2, 64, 16).transpose(1, 2), z(3, dtype=I32)), 1, "w must be contiguous"),
    (lambda: moe.grouped_matmul(z(4, 64), z(16, 64), z(3, dtype=I32)), 1, "w must be a 3-D"),
    (lambda: moe.grouped_matmul(z(4, 64, dtype=F32), z(2, 16, 64), z(3, dtype=I32)), 1, "x must be torch.bfloat16"),
    (lambda: moe.grouped_matmul(z(4, 64), z(2, 16, 64), z(3, dtype=I32), out=z(4, 16, dtype=F32)), 1,
     "out must be torch.bfloat16"),
    (lambda: moe.grouped_matmul(z(4, 64), z(2, 16, 64), z(3, dtype=I32)), 1, "must be on a GPU"),
    (lambda: moe.grouped_matmul_backward(z(4, 64), z(4, 64), z(2, 16, 64), z(3, dtype=I32)), 1, "dy must be [rows, 16]"),
    (lambda: moe.grouped_matmul_backward(z(4, 16), z(3, 64), z(2, 16, 64), z(3, dtype=I32)), 1, "x must have dy's 4 rows"),
    (lambda: moe.grouped_matmul_backward(z(4, 16), z(4, 64), z(2, 16, 64), z(3, dtype=I32), dw_dtype=torch.float16), 1,
     "dw_dtype must be"),
    (lambda: moe.grouped_matmul_backward(z(4, 16), z(4, 64), z(2, 16, 64), z(3, dtype=I32), dx=z(3, 64)), 1,
     "dx must have shape (4, 64)"),
    (lambda: moe.grouped_matmul_backward(z(4, 16), z(4, 64), z(2, 16, 64), z(3, dtype=I32), dx=z(4, 64), need_dx=False),
     1, "dx is given, but need_dx is False"),
    (lambda: moe.grouped_matmul_backward(z(4, 16), None, z(2, 16, 64), z(3, dtype=I32), dw=z(2, 16, 64), need_dw=False),
     1, "dw is given, but need_dw is False"),
])
def test_binding_refusals(lib, call, status, needle):
    with pytest.raises(moe.MoeError) as ei:
        call()
    assert ei.value.status == status and needle in ei.value.message, ei.value.message


def test_binding_refuses_overlapping_outputs(lib):
    x = z(8, 64)
    with pytest.raises(moe.MoeError, match="out must not overlap x"):
        moe.grouped_matmul(x, z(2, 64, 64), z(3, dtype=I32), out=x)
    w = z(2, 64, 64)
    with pytest.raises(moe.MoeError, match="dw must not overlap w"):
        moe.grouped_matmul_backward(z(4, 64), z(4, 64), w, z(3, dtype=I32), dw=w)
    # disjoint halves of one buffer are fine as far as the memory goes
    both = z(8, 64)
    with pytest.raises(moe.MoeError, match="must be on a GPU"):
        moe.grouped_matmul(both[:4], z(2, 64, 64), z(3, dtype=I32), out=both[4:])


BIG = 1 << 32                       # sizes reach the C entries as int32, where BIG + n would count as n


def m(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("call,needle", [
    (lambda: moe.mxfp4_quantize(m(1, BIG + 32)), f"cols={BIG + 32}"),
    (lambda: moe.mxfp4_quantize(m(BIG + 1, 32, dtype=F32)), f"rows={BIG + 1}"),
    (lambda: moe.mxfp4_dequantize(m(1, BIG // 2 + 16, dtype=U8), m(1, BIG // 32 + 1, dtype=U8)), f"cols={BIG + 32}"),
    (lambda: moe.mxfp4_dequantize(m(1, BIG // 4, dtype=U8), m(1, BIG // 64, dtype=U8)), f"cols={BIG // 2}"),
    (lambda: moe.mxfp4_matmul(m(1, 16, dtype=U8), m(1, 1, dtype=U8), m(BIG + 3, 16, dtype=U8), m(BIG + 3, 1, dtype=U8)),
     f"rows={BIG + 3}"),
    (lambda: moe.mxfp4_matmul(*[m(1, (BIG + 64) // d, dtype=U8) for d in (2, 32, 2, 32)]), f"cols={BIG + 64}"),
    (lambda: moe.grouped_matmul(m(BIG + 8, 8), m(1, 8, 8), m(2, dtype=I32)), f"rows={BIG + 8}"),
    (lambda: moe.grouped_matmul(m(4, 8), m(1, BIG + 8, 8), m(2, dtype=I32)), f"n={BIG + 8}"),
    (lambda: moe.grouped_matmul(m(4, BIG + 8), m(1, 8, BIG + 8), m(2, dtype=I32)), f"k={BIG + 8}"),
    (lambda: moe.grouped_matmul_backward(m(BIG + 8, 8), m(BIG + 8, 8), m(1, 8, 8), m(2, dtype=I32)), f"rows={BIG + 8}"),
    (lambda: moe.grouped_matmul_backward(m(4, 8), m(4, 8), m(BIG, 8, 8), m(BIG + 1, dtype=I32)), f"num_groups={BIG}"),
    (lambda: moe.mxfp8_quantize(m(1, BIG + 32)), f"cols={BIG + 32}"),
    (lambda: moe.router_topk(m(BIG + 1, 8, dtype=F32), 2), f"num_tokens={BIG + 1}"),
])
def test_sizes_that_no_int32_holds_are_refused(lib, call, needle):
    with pytest.raises(moe.MoeError) as ei:
        call()
    assert ei.value.status == 2 and needle in ei.value.message, ei.value.message


def test_the_largest_int32_sizes_reach_the_entries_checks(lib):
    """Sizes that an int32 holds are refused, or not, by the entries themselves."""
    most = (1 << 31) - 32
    with pytest.raises(moe.MoeError, match="must be on a GPU"):
        moe.mxfp4_quantize(m(1, most))
    with pytest.raises(moe.MoeError, match="must be on a GPU"):
        moe.mxfp4_dequantize(m(1, most // 2, dtype=U8), m(1, most // 32, dtype=U8))
    with pytest.raises(moe.MoeError, match="must be on a GPU"):
        moe.grouped_matmul(m(most, 8), m(1, 8, 8), m(2, dtype=I32))


def test_the_stride_of_a_matrix_that_is_not_read_is_not_checked(lib):
    """x is read for dw only: without dw it may be NULL, whatever ldx says."""
    no_dw = lambda ldx: (None, 16, None, ldx, P, P, 0, 2, 16, 64, None, None, 0, None, 0, None)
    assert [lib.moe_grouped_matmul_backward(*no_dw(ldx)) for ldx in (0, -8, 3, 64)] == [0] * 4
    refused(lib, "moe_grouped_matmul_backward", (P, 16, P, 0, P, P, 4, 2, 16, 64, None, P, 0, None, 0, None), 2, "ldx must be")


@pytest.mark.parametrize("leaf", ["x", "w"])
def test_a_gradient_that_would_be_lost_is_warned_of(lib, leaf):
    """grouped_matmul records no graph: where autograd would have, it says so."""
    t = {"x": z(4, 64), "w": z(2, 16, 64)}
    t[leaf].requires_grad_()

    def call():
        with pytest.raises(moe.MoeError, match="must be on a GPU"):
            moe.grouped_matmul(t["x"], t["w"], z(3, dtype=I32))

    with pytest.warns(UserWarning, match="grouped_matmul records no autograd graph") as seen:
        call()
    assert seen[0].filename == __file__
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with torch.no_grad():
            call()
        t[leaf].requires_grad_(False)
        call()


def test_the_binding_asks_for_every_workspace_there_is(lib):
    """Sums that the binding takes to be whole are: no workspace for any of them, while one
    is given not far above (the binding's limit is the entries' rule, not a looser one)."""
    fwd, bwd = lib.moe_grouped_matmul_workspace, lib.moe_grouped_matmul_backward_workspace
    most = moe._LONGEST_WHOLE_SUM
    lengths = list(range(8, most + 1, 8))
    for rows, groups, other in ((1, 1, 8), (1, 4096, 8), (64, 1, 128), (300, 2, 512), (4000, 1, 64), (700, 40, 8192)):
        assert not any(fwd(rows, groups, other, length) for length in lengths), (rows, groups, other)
        assert not any(bwd(rows, groups, length, other, 1, 0) for length in lengths), (rows, groups, other)
    for groups, n, k in ((1, 8, 8), (1, 584, 184), (7, 128, 128), (64, 64, 64)):
        assert not any(bwd(rows * groups, groups, n, k, 0, 1) for rows in lengths), (groups, n, k)
    near = most + most // 10
    assert fwd(64, 1, 64, near // 8 * 8) and bwd(64, 1, near // 8 * 8, 64, 1, 0) and bwd(2 * near, 2, 64, 64, 0, 1)
