"""GPU tests of the MXFP4 quantiser and product and of the grouped products,
against the fp64 definitions.

Where inputs are small integers (or MXFP4 codes with scales within a few powers
of two), every partial sum is a multiple of one power of two below 2^24 of it:
fp32 sums are then exact in any order and the output has one right bit pattern,
the nearest-even rounding of the exact value.  Those tests compare bits.

With real-valued inputs an fp32 sum of n products is off by at most
n 2^-23 sum|a b| (one rounding or truncation of at most 2^-23 relative per
addition), then half a bf16 step, 2^-8 of the value, where it is rounded.
"""
import os
import sys

import numpy as np
import pytest
import torch

import oracle
import mxfp4_routed_expert_topk_amd as moe

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.load_library()


def dev():
    return torch.device("cuda:0")


def up(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(dev())
    return t if dtype is None else t.to(dtype)


def f64(t):
    return t.double().cpu().numpy()


def bf16_rounded(v):
    """Nearest-even bf16 of fp64 values that fp32 holds exactly."""
    f = np.asarray(v, np.float64).astype(np.float32)
    assert (f.astype(np.float64) == v).all()
    return oracle.bf16_bits_to_f64(oracle.f32_to_bf16_rne(f))


# ------------------------------------------------------------------ quantiser
def quant_input(rows, cols, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-20, 20, (rows, 1)))
    b = x.reshape(rows, cols // 32, 32)
    kind = rng.random(b.shape[:2])
    b[kind < 0.1] = 0.0
    b[(kind >= 0.1) & (kind < 0.2)] *= 2.0 ** -130          # subnormal or nothing at all
    b[(kind >= 0.2) & (kind < 0.25), 7] = np.inf
    b[(kind >= 0.25) & (kind < 0.3), 31] = np.nan
    # every grid value and every tie, at a scale of its own
    grid = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7])
    ties = kind >= 0.7
    n = int(ties.sum())
    b[ties] = np.concatenate([grid, -grid]) * np.exp2(rng.integers(-120, 120, (n, 1)))
    return x


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (5, 2048), (64, 7168), (1000, 160), (1, 16384)])
def test_quantize_is_exact(rows, cols, dtype):
    x = up(quant_input(rows, cols, rows + cols).astype(np.float32)).to(dtype)
    codes, scales = moe.mxfp4_quantize(x)
    want_c, want_s = oracle.mxfp4_quantize(f64(x))
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)
    np.testing.assert_array_equal(codes.cpu().numpy(), want_c)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_quantize_extremes(dtype):
    """The type's largest and smallest magnitudes: bytes stay in 2..252."""
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).tiny
    x = torch.zeros((6, 32), dtype=dtype, device=dev())
    x[0, :3] = torch.tensor([big, -big, big / 3], dtype=dtype)
    x[1, :3] = torch.tensor([tiny, -tiny, tiny / 2], dtype=dtype)
    x[2, 0] = 2.0 ** -133
    x[3, :2] = torch.tensor([big, tiny], dtype=dtype)
    x[4, :4] = torch.tensor([2.0 ** -123, 2.0 ** -125, 1.5 * 2.0 ** -127, 2.0 ** -127], dtype=dtype)
    codes, scales = moe.mxfp4_quantize(x)
    want_c, want_s = oracle.mxfp4_quantize(f64(x))
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)
    np.testing.assert_array_equal(codes.cpu().numpy(), want_c)
    assert want_s.max() == 252 and want_s.min() == 2


@pytest.mark.parametrize("dtype,pad", [(BF, 8), (BF, 64), (torch.float32, 4), (torch.float32, 12)])
def test_quantize_rows_of_a_wider_matrix(dtype, pad):
    wide = up(quant_input(37, 96, 5).astype(np.float32)).to(dtype)
    base = torch.full((37, 96 + pad), float("nan"), dtype=dtype, device=dev())
    base[:, :96] = wide
    codes = torch.empty((37, 48), dtype=torch.uint8, device=dev())
    scales = torch.empty((37, 3), dtype=torch.uint8, device=dev())
    got = moe.mxfp4_quantize(base[:, :96], codes=codes, scales=scales)
    assert got[0] is codes and got[1] is scales
    want = moe.mxfp4_quantize(wide)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (8, 256), (333, 2048), (2080, 8192)])
def test_dequantize_is_exact(rows, cols, dtype):
    """Every byte 0..255 occurs: 0 is 2^-127, 254 overflows for codes 4 and 6, 255 is NaN."""
    rng = np.random.default_rng(rows)
    codes = rng.integers(0, 256, (rows, cols // 2), dtype=np.uint8)
    scales = rng.integers(0, 256, (rows, cols // 32), dtype=np.uint8)
    scales.reshape(-1)[:4] = [0, 1, 254, 255][:scales.size]
    v = oracle.mxfp4_values(codes, scales)
    v = np.where(np.abs(v) >= 2.0 ** 128, np.copysign(np.inf, v), v)
    got = moe.mxfp4_dequantize(up(codes), up(scales), dtype=dtype)
    assert got.dtype == dtype
    np.testing.assert_array_equal(f64(got), v)
    out = torch.empty((rows, cols), dtype=dtype, device=dev())
    assert moe.mxfp4_dequantize(up(codes), up(scales), out=out) is out
    np.testing.assert_array_equal(f64(out), v)


# ------------------------------------------------------------------ product
def mx_operand(rng, rows, k, low=126, high=129):
    return (rng.integers(0, 256, (rows, k // 2), dtype=np.uint8),
            rng.integers(low, high, (rows, k // 32), dtype=np.uint8))


MATMUL_SIZES = [(1, 1, 32), (1, 16, 64), (2, 17, 96), (16, 16, 128), (17, 33, 160), (1, 4096, 1024), (5, 100, 2048),
                (33, 257, 288), (64, 64, 512), (65, 130, 544), (128, 128, 256), (130, 250, 1056), (256, 256, 768),
                (257, 511, 800), (300, 1000, 2048), (513, 264, 4096), (700, 300, 96), (1, 129, 4128), (37, 384, 1376),
                (3585, 3601, 160), (3401, 3704, 1056),   # 256 x 256 tiles
                (1500, 1201, 1056), (1500, 1208, 800), (1500, 1204, 352), (2000, 640, 512),   # 128 x 128
                (17, 4101, 160), (50, 2101, 1056), (64, 2100, 2048)]   # two and four row blocks a workgroup


@pytest.mark.parametrize("m,n,k", MATMUL_SIZES)
def test_matmul_is_exact(m, n, k):
    """Scale bytes 126..128: products are multiples of 2^-4 and a sum stays below
    36 * 4 * 4128 < 2^20, so every fp32 sum is exact."""
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    a, b = mx_operand(rng, m, k), mx_operand(rng, n, k)
    want = oracle.mxfp4_matmul(*a, *b)
    args = [up(t) for t in (*a, *b)]
    np.testing.assert_array_equal(f64(moe.mxfp4_matmul(*args, dtype=torch.float32)), want)
    got = moe.mxfp4_matmul(*args)
    assert got.dtype == BF
    np.testing.assert_array_equal(f64(got), bf16_rounded(want))


@pytest.mark.parametrize("m,n,k", [(3, 40, 7168), (190, 200, 2048), (600, 512, 7168)])
def test_matmul_of_spread_scales(m, n, k):
    rng = np.random.default_rng(k + m)
    a, b = mx_operand(rng, m, k, 110, 145), mx_operand(rng, n, k, 110, 145)
    want = oracle.mxfp4_matmul(*a, *b)
    size = np.abs(oracle.mxfp4_values(*a)) @ np.abs(oracle.mxfp4_values(*b)).T
    args = [up(t) for t in (*a, *b)]
    # blocks of 32 are exact: one addition per block, plus those inside an instruction
    bound = (k / 32 + 4) * 2.0 ** -23 * size
    got = f64(moe.mxfp4_matmul(*args, dtype=torch.float32))
    assert (np.abs(got - want) <= bound).all()
    got = f64(moe.mxfp4_matmul(*args))
    assert (np.abs(got - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound)).all()


@pytest.mark.parametrize("m,n", [(4, 20), (300, 280)])
def test_matmul_nan_and_edge_scales(m, n):
    """0xFF poisons exactly its row or column; byte 0 is 2^-127; an overflow is an infinity.
    Row 3 and column 7 have scale 2^127 and codes 6: a block's sum there is a multiple of
    3 * 2^127 or 0, so beyond fp32's largest value (below 2^128) unless it cancels within the
    block; block sums of both signs are +inf and -inf and add up to NaN.  Only [3, 7], whose
    blocks are all positive, is sure to be an infinity."""
    k = 352
    rng = np.random.default_rng(m)
    a, b = mx_operand(rng, m, k), mx_operand(rng, n, k)
    a[1][1, 10], b[1][5, 3] = 255, 255
    a[1][2, :] = 0
    a[1][3, :], b[1][7, :] = 254, 254
    a[0][3, :], b[0][7, :] = 0x77, 0x77          # sixes
    want = oracle.mxfp4_matmul(*a, *b)
    got = f64(moe.mxfp4_matmul(*[up(t) for t in (*a, *b)], dtype=torch.float32))
    bad = np.zeros((m, n), bool)
    bad[1], bad[:, 5] = True, True
    assert np.isnan(got[bad]).all()
    assert np.isposinf(got[3, 7])
    other = ~bad
    other[3], other[:, 7] = False, False
    assert np.isfinite(got[other]).all()
    other[2] = False
    np.testing.assert_array_equal(got[other], want[other])
    # row 2 (scale 2^-127): each of at most 11 + 4 additions may flush a subnormal, below 2^-126
    row2 = np.delete(got[2], [5, 7])
    assert (np.abs(row2 - np.delete(want[2], [5, 7])) <= 16 * 2.0 ** -126).all()


# ------------------------------------------------------------------ grouped products
def offsets_of(counts, first=0):
    return np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)


GROUPED = [   # counts, n, k, rows before and behind the groups
    ([1], 8, 8, 0, 0),
    ([0, 1, 0], 8, 64, 0, 0),
    ([3, 0, 2], 40, 72, 2, 5),
    ([16, 1, 17], 128, 128, 0, 1),
    ([32, 31, 33, 0], 136, 200, 1, 0),
    ([64, 65], 64, 520, 0, 9),
    ([127, 0, 128, 129], 256, 256, 0, 0),
    ([300], 264, 136, 3, 3),
    ([255, 257, 1], 248, 320, 0, 40),
    ([0, 0, 0], 64, 64, 0, 4),
    ([700, 5], 384, 576, 0, 0),
    ([2] * 70, 72, 96, 0, 0),
    ([1, 0] * 64 + [9], 128, 64, 0, 2),
    ([513, 40], 520, 1032, 0, 7),
    # enough columns for every tile shape: 256 rows forward, 128 with few rows a group, 128 with many
    ([300, 0, 257], 16392, 72, 0, 3),
    ([20] * 10, 5512, 136, 1, 1),
    ([100, 60], 16392, 40, 0, 0),
    ([130, 0, 7, 260, 33], 2000, 1800, 2, 2),   # 256 x 256 tiles backward
    ([353, 417, 33, 200, 129], 9480, 136, 1, 0),   # 256 x 256 tiles forward, every number of live row blocks
    ([700, 500, 333], 264, 2600, 0, 1),   # 128 x 128 tiles for both gradients
    # long sums for few tiles, in parts: forward, forward of few rows, dw, dx, both gradients
    ([718], 64, 6672, 1, 1),
    ([1, 0, 3, 0, 1, 0] * 3, 264, 5552, 2, 0),
    ([6000], 584, 184, 3, 2),
    ([90, 0, 30], 4104, 72, 2, 1),
    ([3300], 3208, 72, 1, 2),
]


def ints(rng, shape, most=2):
    return rng.integers(-most, most + 1, shape).astype(np.float64)


def grouped_case(counts, n, k, before, behind, seed, most=2):
    rng = np.random.default_rng(seed)
    rows = before + sum(counts) + behind
    off = offsets_of(counts, before)
    x, dy, w = ints(rng, (rows, k), most), ints(rng, (rows, n), most), ints(rng, (len(counts), n, k), most)
    return off, x, dy, w


def poisoned(a, off):
    """Rows outside every group hold NaN."""
    a = a.copy()
    a[:off[0]] = np.nan
    a[off[-1]:] = np.nan
    return a


@pytest.mark.parametrize("counts,n,k,before,behind", GROUPED)
def test_grouped_matmul_is_exact(counts, n, k, before, behind):
    off, x, _, w = grouped_case(counts, n, k, before, behind, n + k)
    out = np.full((len(x), n), 13.0)
    want = oracle.grouped_matmul(x, w, off, out)
    got = up(out, BF)
    assert moe.grouped_matmul(up(poisoned(x, off), BF), up(w, BF), up(off), out=got) is got
    np.testing.assert_array_equal(f64(got), bf16_rounded(want))


@pytest.mark.parametrize("dw_dtype", [BF, torch.float32])
@pytest.mark.parametrize("counts,n,k,before,behind", GROUPED)
def test_grouped_backward_is_exact(counts, n, k, before, behind, dw_dtype):
    off, x, dy, w = grouped_case(counts, n, k, before, behind, abs(n - k))
    keep = np.full((len(x), k), -3.0)
    want_dx, want_dw = oracle.grouped_matmul_backward(dy, x, w, off, keep)
    dx = up(keep, BF)
    dw = torch.full(w.shape, float("nan"), dtype=dw_dtype, device=dev())
    got = moe.grouped_matmul_backward(up(poisoned(dy, off), BF), up(poisoned(x, off), BF), up(w, BF), up(off), dx=dx, dw=dw)
    assert got[0] is dx and got[1] is dw
    np.testing.assert_array_equal(f64(dx), bf16_rounded(want_dx))
    np.testing.assert_array_equal(f64(dw), want_dw if dw_dtype == torch.float32 else bf16_rounded(want_dw))


def test_grouped_one_gradient_only():
    off, x, dy, w = grouped_case([5, 9], 48, 80, 0, 0, 1)
    args = [up(t, BF) for t in (dy, x, w)] + [up(off)]
    dx, dw = moe.grouped_matmul_backward(*args)
    assert dw.dtype == torch.float32
    only_dx = moe.grouped_matmul_backward(args[0], None, args[2], args[3], need_dw=False)
    only_dw = moe.grouped_matmul_backward(*args, need_dx=False)
    assert only_dx[1] is None and torch.equal(only_dx[0], dx)
    assert only_dw[0] is None and torch.equal(only_dw[1], dw)


@pytest.mark.parametrize("counts,n,k", [([718], 64, 6672), ([1, 0, 3] * 6, 264, 5552), ([6000, 566], 584, 184),
                                        ([90, 30], 4104, 72), ([3300], 3208, 72)])
def test_grouped_sums_in_parts_and_whole(counts, n, k):
    """With and without a workspace, of sums that are exact: the same bits."""
    off, x, dy, w = grouped_case(counts, n, k, 0, 0, 8)
    X, DY, W, O = up(x, BF), up(dy, BF), up(w, BF), up(off)
    lib, rows, G = moe.load_library(), len(x), len(counts)
    assert lib.moe_grouped_matmul_workspace(rows, G, n, k) + \
        lib.moe_grouped_matmul_backward_workspace(rows, G, n, k, 1, 1) > 0
    y, dx, dw = torch.zeros_like(DY), torch.zeros_like(X), torch.zeros(W.shape, device=dev())
    s = torch.cuda.current_stream().cuda_stream
    assert lib.moe_grouped_matmul(X.data_ptr(), k, W.data_ptr(), O.data_ptr(), rows, G, n, k, y.data_ptr(), None, 0, s) == 0
    assert lib.moe_grouped_matmul_backward(DY.data_ptr(), n, X.data_ptr(), k, W.data_ptr(), O.data_ptr(), rows, G, n, k,
                                           dx.data_ptr(), dw.data_ptr(), moe.MOE_F32, None, 0, s) == 0
    got = moe.grouped_matmul(X, W, O), *moe.grouped_matmul_backward(DY, X, W, O)
    for g, t in zip(got, (y, dx, dw)):
        assert torch.equal(g, t)


PARTS = [([718], 64, 6672), ([1, 0, 3] * 6, 264, 5552), ([90, 30], 4104, 72), ([3300], 3208, 72), ([6000, 566], 584, 184)]


@pytest.mark.parametrize("counts,n,k", PARTS)
def test_grouped_sums_in_parts_of_real_values(counts, n, k):
    """A sum in parts has no more additions, one after another, than the whole one: the same bounds."""
    rng = np.random.default_rng(n)
    off = offsets_of(counts)
    rows = int(off[-1])
    assert moe.load_library().moe_grouped_matmul_workspace(rows, len(counts), n, k) + \
        moe.load_library().moe_grouped_matmul_backward_workspace(rows, len(counts), n, k, 1, 1) > 0
    x, dy = (torch.from_numpy(rng.standard_normal((rows, c)) * np.exp2(rng.integers(-6, 7, (rows, 1)))).to(BF) for c in (k, n))
    w = torch.from_numpy(rng.standard_normal((len(counts), n, k)) / 40).to(BF)
    X, DY, W = f64(x), f64(dy), f64(w)
    y = moe.grouped_matmul(x.to(dev()), w.to(dev()), up(off))
    dx, dw = moe.grouped_matmul_backward(dy.to(dev()), x.to(dev()), w.to(dev()), up(off))
    zero = lambda c: np.zeros((rows, c))
    want = oracle.grouped_matmul(X, W, off, zero(n)), *oracle.grouped_matmul_backward(DY, X, W, off, zero(k))
    size = (oracle.grouped_matmul(abs(X), abs(W), off, zero(n)),
            *oracle.grouped_matmul_backward(abs(DY), abs(X), abs(W), off, zero(k)))
    for name, got, ref, big, terms in (("y", y, want[0], size[0], k), ("dx", dx, want[1], size[1], n),
                                       ("dw", dw, want[2], size[2], max(counts))):
        bound = terms * 2.0 ** -23 * big
        if got.dtype == BF:
            bound = bound + 2.0 ** -8 * (abs(ref) + bound)
        assert (abs(f64(got) - ref) <= bound).all(), name


@pytest.mark.parametrize("dw_dtype", [BF, torch.float32])
@pytest.mark.parametrize("counts,n,k", [([6600, 0], 584, 184), ([9700, 0, 30], 64, 184), ([0, 6600], 40, 72)])
def test_grouped_weight_gradients_in_parts_of_an_empty_group(counts, n, k, dw_dtype):
    """Parts without rows still give zeros: dw held NaN."""
    off, x, dy, w = grouped_case(counts, n, k, 1, 2, 5)
    assert moe.load_library().moe_grouped_matmul_backward_workspace(len(x), len(counts), n, k, 0, 1) > 0
    dw = torch.full(w.shape, float("nan"), dtype=dw_dtype, device=dev())
    moe.grouped_matmul_backward(up(poisoned(dy, off), BF), up(poisoned(x, off), BF), up(w, BF), up(off), dw=dw, need_dx=False)
    want = oracle.grouped_matmul_backward(dy, x, w, off, np.zeros(x.shape))[1]
    np.testing.assert_array_equal(f64(dw), want if dw_dtype == torch.float32 else bf16_rounded(want))


@pytest.mark.parametrize("counts,n,k", PARTS)
def test_grouped_sums_in_parts_on_another_stream(counts, n, k):
    """The workspace is the given stream's, the inputs are kept until it has passed: neither is
    given to what either stream allocates right after the call."""
    off, x, dy, w = grouped_case(counts, n, k, 0, 0, 21)
    X, DY, W, O = up(x, BF), up(dy, BF), up(w, BF), up(off)
    want = moe.grouped_matmul(X, W, O), *moe.grouped_matmul_backward(DY, X, W, O)
    busy = torch.ones((4096, 4096), dtype=BF, device=dev())
    sizes = {t.numel() for t in (X, DY, W, O)} | {want[2].numel() * 8, 1 << 19, 1 << 21}
    s = torch.cuda.Stream()
    for _ in range(3):
        args = [t.clone() for t in (DY, X, W, O)]
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(4):
                torch.mm(busy, busy)
        got = moe.grouped_matmul(*args[1:], stream=s), *moe.grouped_matmul_backward(*args, stream=s)
        del args
        junk = [torch.full((m,), float("nan"), device=dev()) for m in sizes]
        with torch.cuda.stream(s):
            junk += [torch.full((m,), float("nan"), device=dev()) for m in sizes]
        torch.cuda.current_stream().wait_stream(s)
        for g, t in zip(got, want):
            assert torch.equal(g, t)
        del junk, got


def test_grouped_sums_in_parts_in_a_graph():
    off, x, dy, w = grouped_case([90, 30], 4104, 72, 1, 1, 9)
    X, DY, W, O = up(x, BF), up(dy, BF), up(w, BF), up(off)
    wt = W.transpose(1, 2).contiguous()
    step = lambda: (moe.grouped_matmul(DY, wt, O), *moe.grouped_matmul_backward(DY, X, W, O))
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = step()
    for turn in range(3):
        DY.copy_(up(ints(np.random.default_rng(turn), dy.shape), BF))
        want = [t.clone() for t in step()]
        for t in res:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for got, ref in zip(res, want):
            lo, hi = (1, 121) if got.dim() == 2 else (0, None)   # the first and last rows are no group's
            assert torch.equal(got[lo:hi], ref[lo:hi])


@pytest.mark.parametrize("counts,n,k", [([700, 500, 333], 264, 2600), ([353, 417, 33, 200, 129], 136, 9480)])
def test_grouped_one_gradient_in_other_tiles(counts, n, k):
    """A gradient alone may take other tiles than both: the sums are the same."""
    off, x, dy, w = grouped_case(counts, n, k, 0, 0, 4)
    args = [up(t, BF) for t in (dy, x, w)] + [up(off)]
    dx, dw = moe.grouped_matmul_backward(*args)
    assert torch.equal(moe.grouped_matmul_backward(args[0], None, args[2], args[3], need_dw=False)[0], dx)
    assert torch.equal(moe.grouped_matmul_backward(*args, need_dx=False)[1], dw)
    np.testing.assert_array_equal(f64(dx), bf16_rounded(oracle.grouped_matmul_backward(dy, x, w, off, np.zeros(x.shape))[0]))


@pytest.mark.parametrize("counts,n,k", [([40, 0, 90], 256, 1024), ([700, 3, 41], 520, 2048), ([5, 0, 1, 17], 512, 7168)])
def test_grouped_of_real_values(counts, n, k):
    rng = np.random.default_rng(k)
    off = offsets_of(counts)
    rows = int(off[-1])
    x, dy = (torch.from_numpy(rng.standard_normal((rows, c))).to(BF) for c in (k, n))
    w = torch.from_numpy(rng.standard_normal((len(counts), n, k)) / 40).to(BF)
    X, DY, W = f64(x), f64(dy), f64(w)
    y = moe.grouped_matmul(x.to(dev()), w.to(dev()), up(off))
    dx, dw = moe.grouped_matmul_backward(dy.to(dev()), x.to(dev()), w.to(dev()), up(off))
    zero = lambda c: np.zeros((rows, c))
    want = oracle.grouped_matmul(X, W, off, zero(n)), *oracle.grouped_matmul_backward(DY, X, W, off, zero(k))
    size = (oracle.grouped_matmul(abs(X), abs(W), off, zero(n)),
            *oracle.grouped_matmul_backward(abs(DY), abs(X), abs(W), off, zero(k)))
    for name, got, ref, big, terms in (("y", y, want[0], size[0], k), ("dx", dx, want[1], size[1], n),
                                       ("dw", dw, want[2], size[2], max(counts))):
        bound = terms * 2.0 ** -23 * big
        if got.dtype == BF:
            bound = bound + 2.0 ** -8 * (abs(ref) + bound)
        assert (abs(f64(got) - ref) <= bound).all(), name
        if got.dtype == BF:   # rounding alone: 2^-8 of every value, and so of the norm; the sums add far less
            assert np.linalg.norm(f64(got) - ref) <= 2.0 ** -8 * np.linalg.norm(ref), name


def test_grouped_gradients_are_differences_of_the_product():
    """With small integers every product is exact: sum(dy * (f(x+u) - f(x-u))) / 2 is
    sum(dx * u) to the last bit, and the same for w."""
    rng = np.random.default_rng(8)
    counts, n, k = [9, 0, 33], 40, 56
    off, x, dy, w = grouped_case(counts, n, k, 0, 0, 8, most=1)
    ux, uw = ints(rng, x.shape, 1), ints(rng, w.shape, 1)
    f = lambda x, w: f64(moe.grouped_matmul(up(x, BF), up(w, BF), up(off)))
    dx, dw = moe.grouped_matmul_backward(up(dy, BF), up(x, BF), up(w, BF), up(off))
    # |y| <= 56 * 2: exact in bf16
    assert (dy * (f(x + ux, w) - f(x - ux, w))).sum() / 2 == (f64(dx) * ux).sum()
    assert (dy * (f(x, w + uw) - f(x, w - uw))).sum() / 2 == (f64(dw) * uw).sum()


def test_grouped_row_strides():
    off, x, dy, w = grouped_case([20, 45], 72, 88, 1, 2, 4)
    rows = len(x)
    wide_x = torch.full((rows, 88 + 24), float("nan"), dtype=BF, device=dev())
    wide_dy = torch.full((rows, 2 * 72), float("nan"), dtype=BF, device=dev())
    wide_x[:, 8:96], wide_dy[:, 72:] = up(x, BF), up(dy, BF)
    args = wide_dy[:, 72:], wide_x[:, 8:96], up(w, BF), up(off)
    out, dx = torch.zeros((rows, 72), dtype=BF, device=dev()), torch.zeros((rows, 88), dtype=BF, device=dev())
    moe.grouped_matmul(args[1], args[2], args[3], out=out)
    _, dw = moe.grouped_matmul_backward(*args, dx=dx)
    want_dx, want_dw = oracle.grouped_matmul_backward(dy, x, w, off, np.zeros((rows, 88)))
    np.testing.assert_array_equal(f64(out), bf16_rounded(oracle.grouped_matmul(x, w, off, np.zeros((rows, 72)))))
    np.testing.assert_array_equal(f64(dx), bf16_rounded(want_dx))
    np.testing.assert_array_equal(f64(dw), want_dw)


def test_grouped_masked_values_stay_in_their_row():
    """NaN and infinities in one group's rows reach that group's outputs only."""
    off, x, dy, w = grouped_case([30, 70, 30], 136, 200, 0, 0, 6)
    x[40, 3], dy[50, 7] = np.inf, np.nan
    args = up(dy, BF), up(x, BF), up(w, BF), up(off)
    y = f64(moe.grouped_matmul(args[1], args[2], args[3]))
    dx, dw = (f64(t) for t in moe.grouped_matmul_backward(*args))
    assert np.isfinite(np.delete(y, 40, axis=0)).all() and not np.isfinite(y[40]).all()
    assert np.isfinite(np.delete(dx, 50, axis=0)).all() and np.isnan(dx[50]).all()
    assert np.isfinite(dw[[0, 2]]).all()
    bad = ~np.isfinite(dw[1])
    assert bad[7].all() and bad[:, 3].all() and bad.sum() == 200 + 136 - 1


def test_grouped_offsets_are_clamped():
    """Offsets outside [0, rows] or decreasing reach no other memory: they act clamped."""
    _, x, dy, w = grouped_case([8] * 4, 64, 72, 0, 0, 2)
    off = np.array([-5, 8, 40, 30, 1 << 30], np.int32)      # groups 0..8, 8..32, empty, 30..32
    y = torch.zeros((32, 64), dtype=BF, device=dev())
    moe.grouped_matmul(up(x, BF), up(w, BF), up(off), out=y)
    _, dw = moe.grouped_matmul_backward(up(dy, BF), up(x, BF), up(w, BF), up(off), need_dx=False)
    np.testing.assert_array_equal(f64(y)[:30], oracle.grouped_matmul(x, w, [0, 8, 30, 30, 30], np.zeros((32, 64)))[:30])
    want = np.stack([dy[:8].T @ x[:8], dy[8:].T @ x[8:], np.zeros((64, 72)), dy[30:].T @ x[30:]])
    np.testing.assert_array_equal(f64(dw), want)


DECREASING = [   # offsets (the largest is the number of rows), n, k
    ([0, 718, 0, 718], 64, 6672),               # the forward sum in parts
    ([0, 400, 300, 600, 718], 64, 6672),
    ([50, 100, 0, 120, 90, 130], 4104, 72),     # dx in parts
    ([0, 6000, 10, 9700], 584, 184),
    ([7, 3, 260, 255, 255, 400, 0, 401], 264, 136),
    (list(range(0, 900, 3)) + [40, 41, 800, 905, 899, 910, 0, 912], 72, 96),   # several groups a lane
    (list(range(900, 0, -3)), 72, 96),
]


@pytest.mark.parametrize("offsets,n,k", DECREASING)
def test_grouped_decreasing_offsets_share_no_row(offsets, n, k):
    """An offset below an earlier one counts as that one: in out and dx every row is the first
    group's that holds it, whole, and the same in every run; dw takes each pair as it is."""
    rng = np.random.default_rng(len(offsets) + k)
    rows, groups = max(offsets), len(offsets) - 1
    x, dy, w = ints(rng, (rows + 3, k)), ints(rng, (rows + 3, n)), ints(rng, (groups, n, k))
    # the rows behind the largest offset are no group's
    off = np.maximum.accumulate(offsets)
    Y, D = np.full((rows + 3, n), 11.0), np.full((rows + 3, k), -7.0)
    args = up(dy, BF), up(x, BF), up(w, BF), up(np.array(offsets, np.int32))
    want_y = bf16_rounded(oracle.grouped_matmul(x, w, off, Y))
    want_dx = bf16_rounded(oracle.grouped_matmul_backward(dy, x, w, off, D)[0])
    want_dw = np.stack([dy[i:max(i, j)].T @ x[i:max(i, j)] for i, j in zip(offsets, offsets[1:])])
    for _ in range(2):
        np.testing.assert_array_equal(f64(moe.grouped_matmul(*args[1:], out=up(Y, BF))), want_y)
        dx, dw = moe.grouped_matmul_backward(*args, dx=up(D, BF))
        np.testing.assert_array_equal(f64(dx), want_dx)
        np.testing.assert_array_equal(f64(dw), want_dw)


def test_grouped_empty_calls():
    w = torch.ones((3, 16, 24), dtype=BF, device=dev())
    off = torch.zeros(4, dtype=torch.int32, device=dev())
    e = lambda c: torch.empty((0, c), dtype=BF, device=dev())
    assert moe.grouped_matmul(e(24), w, off).shape == (0, 16)
    dx, dw = moe.grouped_matmul_backward(e(16), e(24), w, off)
    assert dx.shape == (0, 24) and (dw == 0).all()
    none = torch.empty((0, 16, 24), dtype=BF, device=dev())
    y = torch.full((2, 16), 5.0, dtype=BF, device=dev())
    moe.grouped_matmul(torch.ones((2, 24), dtype=BF, device=dev()), none, off[:1], out=y)
    assert (y == 5).all()
    x4 = torch.empty((0, 64), device=dev())
    codes, scales = moe.mxfp4_quantize(x4)
    assert codes.shape == (0, 32) and moe.mxfp4_dequantize(codes, scales).shape == (0, 64)
    assert moe.mxfp4_matmul(codes, scales, codes, scales).shape == (0, 0)


@pytest.mark.parametrize("m,n,k", [(20, 300, 1056), (700, 300, 96), (1500, 1204, 352), (3401, 3704, 544)])
def test_mxfp4_rows_of_larger_matrices(m, n, k):
    """A range of rows: its scales may start at any address."""
    rng = np.random.default_rng(k)
    full = [up(t) for t in (*mx_operand(rng, m + 5, k), *mx_operand(rng, n + 6, k))]
    part = [t[c:] for t, c in zip(full, (5, 5, 3, 3))]
    part[2:] = [t[:n] for t in part[2:]]
    assert any(t.data_ptr() % 16 for t in part)
    own = [t.clone() for t in part]
    assert torch.equal(moe.mxfp4_matmul(*part), moe.mxfp4_matmul(*own))
    assert torch.equal(moe.mxfp4_dequantize(*part[:2]), moe.mxfp4_dequantize(*own[:2]))
    x = moe.mxfp4_dequantize(*own[:2])
    full[0].zero_(), full[1].zero_()
    moe.mxfp4_quantize(x, codes=part[0], scales=part[1])
    want = moe.mxfp4_quantize(x)
    assert torch.equal(part[0], want[0]) and torch.equal(part[1], want[1])
    assert not full[0][:5].any() and not full[1][:5].any()


def test_grouped_range_of_groups():
    """Some of the groups, their offsets as they lie in the whole array: the others' rows are left."""
    off, x, dy, w = grouped_case([30, 70, 0, 41, 9], 136, 200, 2, 3, 6)
    X, DY, W, O = up(x, BF), up(dy, BF), up(w, BF), up(off)
    whole = moe.grouped_matmul(X, W, O), *moe.grouped_matmul_backward(DY, X, W, O)
    lo, hi = off[1], off[4]
    y, dx = torch.full_like(whole[0], 7.0), torch.full_like(whole[1], 7.0)
    moe.grouped_matmul(X, W[1:4], O[1:5], out=y)
    _, dw = moe.grouped_matmul_backward(DY, X, W[1:4], O[1:5], dx=dx)
    for got, ref in ((y, whole[0]), (dx, whole[1])):
        assert torch.equal(got[lo:hi], ref[lo:hi]) and bool((got[:lo] == 7).all()) and bool((got[hi:] == 7).all())
    assert torch.equal(dw, whole[2][1:4])


# ------------------------------------------------------------------ beyond 32 bits
# Tensors of more than 2^31 elements (and 2^32 bytes), of which the calls use the
# far end; elsewhere rows belong to no group or hold zeros.
def far_rows(rows, cols, used):
    """bf16 [rows, cols], uninitialised but for small integers in the last `used` rows."""
    t = torch.empty((rows, cols), dtype=BF, device=dev())
    a = ints(np.random.default_rng(rows + cols), (used, cols))
    t[rows - used:] = up(a, BF)
    return t, a


def test_quantize_and_dequantize_far_rows():
    # 2^24 + 32 rows of 1024: more lanes than one launch has threads
    rows, cols = (1 << 24), 1024 + 32
    x = torch.zeros((rows, cols), dtype=BF, device=dev())
    tail = up(ints(np.random.default_rng(0), (70, cols)), BF)
    x[-70:] = tail
    codes, scales = moe.mxfp4_quantize(x)
    del x
    want = moe.mxfp4_quantize(tail)
    assert torch.equal(codes[-70:], want[0]) and torch.equal(scales[-70:], want[1])
    assert not codes[-80:-70].any() and bool((scales[-80:-70] == 2).all())
    for dtype in (BF, torch.float32):
        assert torch.equal(moe.mxfp4_dequantize(codes, scales, dtype=dtype)[-70:], moe.mxfp4_dequantize(*want, dtype=dtype))


def test_quantize_far_strided_rows():
    x, a = far_rows(300000, 8192, 40)      # 2.4e9 elements
    codes, scales = moe.mxfp4_quantize(x[:, 64:128])
    want = moe.mxfp4_quantize(up(a[:, 64:128], BF))
    assert torch.equal(codes[-40:], want[0]) and torch.equal(scales[-40:], want[1])


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_matmul_far_outputs(dtype):
    m, n = 50000, 50001                    # 2.5e9 outputs; rows are not 16-byte aligned
    g = torch.Generator(device=dev()).manual_seed(1)
    a, b = (torch.randint(0, 256, (r, 32), dtype=torch.uint8, device=dev(), generator=g) for r in (m, n))
    sa, sb = (torch.full((r, 2), 127, dtype=torch.uint8, device=dev()) for r in (m, n))
    out = moe.mxfp4_matmul(a, sa, b, sb, dtype=dtype)
    av, bv = (moe.mxfp4_dequantize(t, s, dtype=torch.float32).double() for t, s in ((a[-300:], sa[-300:]), (b, sb)))
    # sums of 64 multiples of 1/4 of at most 36: exact in fp32
    assert torch.equal(out[-300:], (av @ bv.t()).to(dtype))
    del out
    out = moe.mxfp4_matmul(b, sb, a, sa, dtype=dtype)      # 16-byte rows
    assert torch.equal(out[-300:].t(), (moe.mxfp4_dequantize(a, sa, dtype=torch.float32).double() @ bv[-300:].t()).to(dtype))


def test_grouped_far_rows():
    rows, n, k, used = 340000, 7168, 264, 700
    off = up(np.array([rows - used, rows - 300, rows - 300, rows], np.int32))
    split = [0, used - 300, used - 300, used]
    dy, a = far_rows(rows, n, used)        # 2.4e9 elements
    w = ints(np.random.default_rng(2), (3, n, k))
    W = up(w, BF)
    dx, dw = moe.grouped_matmul_backward(dy, torch.ones((rows, k), dtype=BF, device=dev()), W, off)
    np.testing.assert_array_equal(f64(dx[-used:]), bf16_rounded(np.concatenate([a[:400] @ w[0], a[400:] @ w[2]])))
    np.testing.assert_array_equal(f64(dw), np.stack([a[i:j].T @ np.ones((j - i, k)) for i, j in zip(split, split[1:])]))
    # the forward product's far input, and its far output
    wt = np.ascontiguousarray(w.transpose(0, 2, 1))
    y = moe.grouped_matmul(dy, up(wt, BF), off)
    np.testing.assert_array_equal(f64(y[-used:]), f64(dx[-used:]))
    del y, dx
    x, a = far_rows(rows, k, used)
    y = moe.grouped_matmul(x, W, off, out=dy)
    np.testing.assert_array_equal(f64(y[-used:]), bf16_rounded(np.concatenate([a[:400] @ w[0].T, a[400:] @ w[2].T])))


def test_grouped_far_groups():
    groups, n, k, rows = 1160, 1024, 2048, 90        # 2.4e9 weights
    off = np.zeros(groups + 1, np.int32)
    off[-2:] = 50, rows
    rng = np.random.default_rng(3)
    x, dy, w = ints(rng, (rows, k)), ints(rng, (rows, n)), ints(rng, (2, n, k))
    W = torch.empty((groups, n, k), dtype=BF, device=dev())
    W[-2:] = up(w, BF)
    args = up(dy, BF), up(x, BF), W, up(off)
    y = f64(moe.grouped_matmul(args[1], W, args[3]))
    np.testing.assert_array_equal(y, bf16_rounded(np.concatenate([x[:50] @ w[0].T, x[50:] @ w[1].T])))
    for dtype in (torch.float32, BF):
        dx, dw = moe.grouped_matmul_backward(*args, dw_dtype=dtype)
        np.testing.assert_array_equal(f64(dx), bf16_rounded(np.concatenate([dy[:50] @ w[0], dy[50:] @ w[1]])))
        for e, (lo, hi) in ((-2, (0, 50)), (-1, (50, rows))):
            want = dy[lo:hi].T @ x[lo:hi]
            np.testing.assert_array_equal(f64(dw[e]), want if dtype == torch.float32 else bf16_rounded(want))
        assert not dw[:-2].any()


# ------------------------------------------------------------------ streams, graphs, and all of them together
def test_on_another_stream():
    off, x, dy, w = grouped_case([100, 28], 128, 192, 0, 0, 3)
    a = up(dy, BF), up(x, BF), up(w, BF), up(off)
    q = moe.mxfp4_quantize(a[1])
    want = moe.grouped_matmul(a[1], a[2], a[3]), *moe.grouped_matmul_backward(*a), moe.mxfp4_matmul(*q, *q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = (moe.grouped_matmul(a[1], a[2], a[3], stream=s), *moe.grouped_matmul_backward(*a, stream=s),
           moe.mxfp4_matmul(*moe.mxfp4_quantize(a[1], stream=s), *q, stream=s))
    torch.cuda.current_stream().wait_stream(s)
    for g, t in zip(got, want):
        assert torch.equal(g, t)


def test_graph_replay_matches_eager():
    counts, n, k = [70, 0, 130, 56], 256, 384
    off, x, dy, w = grouped_case(counts, n, k, 0, 0, 12)
    X, DY, W, O = up(x, BF), up(dy, BF), up(w, BF), up(off)

    def step():
        y = moe.grouped_matmul(X, W, O)
        dx, dw = moe.grouped_matmul_backward(DY, X, W, O)
        a, b = moe.mxfp4_quantize(X), moe.mxfp4_quantize(W[0])
        return y, dx, dw, moe.mxfp4_matmul(*a, *b), moe.mxfp4_dequantize(*a)

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):      # two graphs of the same calls share nothing
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = step()
        graphs.append((g, res))
    for turn in range(4):
        rng = np.random.default_rng(turn)
        X.copy_(up(ints(rng, x.shape), BF))
        cut = np.sort(rng.integers(0, len(x) + 1, len(counts) - 1))
        O.copy_(up(np.concatenate([[0], cut, [len(x)]]).astype(np.int32)))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        for g, res in graphs:
            for t in res:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            for got, ref in zip(res, want):
                assert torch.equal(got, ref)


def test_quantised_weights_feed_the_layer_and_match_the_unfused_products():
    """bf16 weights -> mxfp4_quantize -> the layer's plan and forward, against the
    same layer from its parts: router, route, grouped products over the
    dequantised weights and a slot-order sum, with h rounded to bf16 as in the
    layer.  The two differ by bf16 roundings of h (and of y in the parts):
    each is within the layer's rule of the fp64 layer over the same weights."""
    T, H, I, E, K = 40, 256, 128, 8, 2
    g = torch.Generator(device=dev()).manual_seed(5)
    rnd = lambda *s: torch.randn(s, device=dev(), generator=g)
    w13, w2 = (rnd(E, 2 * I, H) / 16).to(BF), (rnd(E, H, I) / 11).to(BF)
    q13 = moe.mxfp4_quantize(w13.view(E * 2 * I, H))
    q2 = moe.mxfp4_quantize(w2.view(E * H, I))
    ew = [q13[0].view(E, 2 * I, H // 2), q13[1].view(E, 2 * I, H // 32), q2[0].view(E, H, I // 2),
          q2[1].view(E, H, I // 32)]
    plan = moe.Plan(moe.Config(H, I, E, K, T, moe.MOE_ACT_BF16), *ew)
    x = rnd(T, H).to(BF)
    ids, weights = moe.router_topk(rnd(T, E), K)
    out = plan.forward(x, ids, weights)

    _, offsets, perm, rowpos = plan.route(ids)
    rows = x[perm.long() // K]
    v13 = moe.mxfp4_dequantize(*q13).view(E, 2 * I, H)
    v2 = moe.mxfp4_dequantize(*q2).view(E, H, I)
    gu = moe.grouped_matmul(rows, v13, offsets).float()
    h = (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]).to(BF)
    y = moe.grouped_matmul(h, v2, offsets).float()[rowpos.long().view(T, K)]
    parts = (y * weights[..., None]).sum(1)

    ref = oracle.forward(x.view(torch.int16).cpu().numpy().view(np.uint16), ids.cpu().numpy(), weights.cpu().numpy(),
                         [t.cpu().numpy() for t in ew], E)
    assert oracle.check_rows(f64(out), ref)["pass"]
    # the parts round g, u, h and y to bf16 (2^-8 each, of the value): row errors add up to at most
    # 2^-8 (|g| + |u| + |h| + |y| relative to their own norms) ~ 4 * 2^-8
    rel = np.linalg.norm(f64(parts) - ref, axis=1) / np.linalg.norm(ref, axis=1)
    assert rel.max() <= 4 * 2.0 ** -8
    # the gradients of the same rows: dw of w2 over the route order, against fp64
    dy = rnd(T * K, H).to(BF)
    dx, dw = moe.grouped_matmul_backward(dy, h, v2, offsets)
    want_dx, want_dw = oracle.grouped_matmul_backward(f64(dy), f64(h), f64(v2), offsets.cpu().numpy(), np.zeros((T * K, I)))
    assert np.linalg.norm(f64(dx) - want_dx) <= 2.0 ** -8 * np.linalg.norm(want_dx)
    assert np.linalg.norm(f64(dw) - want_dw) <= 2.0 ** -20 * np.linalg.norm(want_dw)
    # a shared expert beside them: the dense product of quantised activations
    shared = moe.mxfp4_matmul(*moe.mxfp4_quantize(x), *q13)
    want = f64(moe.mxfp4_dequantize(*moe.mxfp4_quantize(x))) @ f64(moe.mxfp4_dequantize(*q13)).T
    assert np.linalg.norm(f64(shared) - want) <= 2.0 ** -8 * np.linalg.norm(want)
