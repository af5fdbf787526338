"""GPU tests of the scored router, of the product with an MXFP4 matrix and of the
experts' combine, against the fp64 definitions.

u = 2^-24 is half a step of fp32.  Ids are compared exactly; computed numbers
with bounds counted from the operations:
  a sum of n terms      (n - 1) u sum|terms|, whatever the order
  expf                  2 u relative, and its argument's rounding u |argument|
  the output's rounding half a step: bf16 2^-8, fp32 2^-24 of the value
Where every term is a multiple of one power of two and sums stay below 2^24 of
it, fp32 sums are exact in any order and the output has one right bit pattern.
"""
import numpy as np
import pytest
import torch

import oracle
import mxfp4_routed_expert_topk_amd as moe

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
U = 2.0 ** -24
INF, NAN = float("inf"), float("nan")
F32_MAX = float(np.finfo(np.float32).max)
SCORE = {"softmax": moe.MOE_SCORE_SOFTMAX, "sigmoid": moe.MOE_SCORE_SIGMOID}


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


def half_step(t):
    return torch.finfo(t.dtype).eps / 2


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == BF else torch.int32)


# ------------------------------------------------------------------ router
def spread(logits):
    """The largest argument of an exponential that does not vanish."""
    l = logits[np.isfinite(logits)]
    return min(float(l.max() - l.min()) + float(np.abs(l).max()), 210.0) if l.size else 0.0


def check_select(logits, k, score="softmax", bias=None, renormalize=True, scale=1.0, **groups):
    """logits: fp32 or bf16 tensor on the device; returns what the entry gave."""
    b = None if bias is None else up(np.asarray(bias, np.float32))
    ids, w = moe.router_select(logits, k, score=SCORE[score], bias=b, renormalize=renormalize, scale=scale, **groups)
    l = f64(logits)
    want_i, want_w = oracle.router_select(l, k, score=score, bias=None if b is None else f64(b),
                                          renormalize=renormalize, scale=scale, **groups)
    np.testing.assert_array_equal(ids.cpu().numpy(), want_i)
    # numerator and denominator: an exponential and its argument each; sums over up to 1024 terms of at most
    # 22 additions in a row; two quotients and the scale
    tol = (2 * spread(l) + 40) * U * np.abs(want_w) + 2.0 ** -125
    assert (np.abs(f64(w) - want_w) <= tol).all(), np.abs(f64(w) - want_w).max()
    return ids, w


def logits_of(rng, T, E, dtype, size=2.0):
    return up((rng.standard_normal((T, E)) * size).astype(np.float32)).to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (5, 8, 2), (4, 63, 32), (2, 64, 1), (7, 65, 8), (3, 128, 6), (2, 200, 9),
                                   (5, 257, 16), (3, 384, 8), (2, 513, 32), (4, 896, 16), (1, 1024, 32)])
def test_select_without_bias(T, E, k, score, renormalize, dtype):
    rng = np.random.default_rng(E + k)
    check_select(logits_of(rng, T, E, dtype), k, score, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 8, 3), (9, 64, 8), (4, 100, 16), (6, 384, 8), (3, 896, 16), (2, 1024, 32)])
def test_select_with_a_bias(T, E, k, score, renormalize, dtype):
    rng = np.random.default_rng(E * k)
    check_select(logits_of(rng, T, E, dtype), k, score, bias=rng.standard_normal(E) * 0.3, renormalize=renormalize)


@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,G,L", [(4, 8, 2, 2, 1), (5, 12, 3, 3, 1), (3, 24, 8, 8, 4), (2, 64, 5, 64, 7), (7, 60, 6, 5, 2),
                                       (3, 384, 8, 8, 4), (2, 896, 16, 7, 3), (2, 1024, 32, 32, 1), (3, 992, 9, 31, 30),
                                       (2, 96, 4, 4, 4)])
def test_select_of_groups(T, E, k, G, L, score, biased, group_top):
    rng = np.random.default_rng(E + G)
    bias = rng.standard_normal(E) * 0.2 if biased else None
    check_select(logits_of(rng, T, E, F32), k, score, bias=bias, num_groups=G, group_limit=L, group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_select_equal_values_in_order_of_their_ids(score, biased):
    """Few distinct logits, so that every row has many ties; -0 and 0 are one value."""
    rng = np.random.default_rng(7)
    for E, k, groups in ((40, 12, {}), (896, 32, {}), (896, 16, dict(num_groups=8, group_limit=3, group_top=2)),
                         (64, 8, dict(num_groups=16, group_limit=4, group_top=1))):
        l = rng.choice([-2.0, -0.0, 0.0, 1.5], (6, E)).astype(np.float32)
        l[0] = 0.25   # all equal: the first ids of the first groups
        bias = rng.choice([0.0, -0.0, 0.5], E) if biased else None
        ids, _ = check_select(up(l), k, score, bias=bias, **groups)
        if not biased:
            assert ids[0].tolist() == list(range(k))


def test_select_saturated_scores():
    """Sigmoids that are 1 in 64 bits tie with a bias and rank by logit without one."""
    l = up(np.array([[100.0, 300.0, 200.0, -400.0, -300.0, 50.0]], np.float32))
    ids, _ = check_select(l, 4, "sigmoid", bias=np.zeros(6), renormalize=False)
    assert ids.tolist() == [[0, 1, 2, 5]]
    ids, _ = check_select(l, 6, "sigmoid", renormalize=False)
    assert ids.tolist() == [[1, 2, 0, 5, 4, 3]]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups", [{}, dict(num_groups=4, group_limit=2, group_top=2),
                                    dict(num_groups=4, group_limit=3, group_top=1)])
def test_select_masks(dtype, score, renormalize, biased, groups):
    """-inf and NaN logits, rows without an expert, fewer experts than slots, one group masked,
    the types' extremes, +inf; a bias of -inf, NaN and +inf."""
    rng = np.random.default_rng(3)
    l = rng.standard_normal((12, 80)).astype(np.float32)
    l[0] = -INF
    l[1] = NAN
    l[2, 1:] = -INF
    l[3, ::3] = NAN
    l[4, 20:40] = -INF
    lowest = -F32_MAX if dtype == F32 else torch.finfo(BF).min
    l[5] = lowest
    l[6, :75] = lowest
    l[7, [3, 50]] = INF
    l[8, 7] = -lowest
    l[9] = -INF
    l[9, [5, 25, 45, 65]] = [1.0, 2.0, 3.0, 4.0]
    l[10, :] = lowest
    l[10, 33] = INF
    bias = None
    if biased:
        bias = rng.standard_normal(80) * 0.1
        bias[[2, 30]] = -INF
        bias[[4, 31]] = NAN
        bias[[60, 41]] = INF
    ids, w = check_select(up(l).to(dtype), 8, score, bias=bias, renormalize=renormalize, **groups)
    assert (ids[:2] == -1).all() and (w[:2] == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [48, 128, 640])
@pytest.mark.parametrize("groups", [{}, dict(num_groups=16, group_limit=5, group_top=2),
                                    dict(num_groups=8, group_limit=7, group_top=1)])
def test_select_extreme_biases(score, E, groups):
    """Biases of the type's extremes and of no size, whose sums two by two pass fp32's range."""
    rng = np.random.default_rng(E)
    l = logits_of(rng, 6, E, F32)
    l[4, : E // 2] = -INF
    for values in ([-F32_MAX, F32_MAX], [-F32_MAX], [F32_MAX], [INF, -INF, 0.0], [INF, F32_MAX, -F32_MAX, 1e-45, -1e-45],
                   [-F32_MAX, -F32_MAX, -F32_MAX, -INF, 0.25]):
        check_select(l, 6, score, bias=rng.choice(values, E), **groups)


@pytest.mark.parametrize("E,near", [(40, 40), (384, 30), (384, 384), (896, 60), (1024, 65)])
@pytest.mark.parametrize("groups", [{}, dict(num_groups=8, group_limit=3, group_top=2),
                                    dict(num_groups=8, group_limit=4, group_top=1)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_select_orders_values_that_fp32_cannot(E, near, groups, score):
    """Biases that bring `near` experts' values within a rounding of fp32 of one another."""
    rng = np.random.default_rng(near + E)
    l = np.repeat(rng.standard_normal((1, E)).astype(np.float32), 5, axis=0)
    s = oracle.scores(l[0], score)
    bias = rng.standard_normal(E) * 0.05 - 2.0
    pick = rng.permutation(E)[:near]
    bias[pick] = (0.9 - s)[pick]
    l[1:] += (rng.standard_normal((4, E)) * 1e-7 * np.abs(l[1:])).astype(np.float32)   # the last bits of some logits
    value = s + bias.astype(np.float32)
    gaps = np.diff(np.sort(value[pick]))
    assert (gaps < 6e-8).mean() > 0.9 and (gaps > 1e-14).mean() > 0.5
    check_select(up(l), 8, score, bias=bias, **groups)


def test_select_grades_groups_by_normalised_scores():
    """Softmax scores without a bias: sums of two that are equal before the division by the row's sum and
    not after it, or the other way round. The best expert of every group has the row's largest logit."""
    rng = np.random.default_rng(17)
    differ = 0
    for G in (3, 5, 6, 7, 12, 24, 33):
        l = np.zeros((60, 2 * G), np.float32)
        l[:, 1::2] = rng.choice([-38.5, -38.0, -37.25, -36.875, -36.75, -36.5, -36.0], (60, G))
        e = np.exp(l.astype(np.float64)).reshape(60, G, 2)

        def best(total):          # the two best groups, equal ones in the order of their numbers
            return np.argsort(-(e / total).sum(2), axis=1, kind="stable")[:, :2]
        # rows whose answer does not hang on the last bit of the row's sum, which goes with its order
        total = e.sum((1, 2), keepdims=True)
        sure = np.array([(best(total * (1 + d)) == best(total)).all(1) for d in (-2.0 ** -52, 2.0 ** -51)]).all(0)
        differ += int((best(np.ones_like(total)) != best(total))[sure, 0].sum())
        for limit in (1, 2):
            check_select(up(l[sure]), 2, num_groups=G, group_limit=limit, group_top=2)
    assert differ > 20
    ids, _ = check_select(up(np.array([[0, -38.5, 0, -38.5, 0, -36.8]], np.float32)), 2, num_groups=3, group_limit=1,
                          group_top=2)
    assert ids.tolist() == [[4, 5]]


def test_select_of_few_lanes_with_experts():
    """Fewer lanes than slots hold an open expert; one lane holds many."""
    l = np.full((4, 1024), -INF, np.float32)
    rng = np.random.default_rng(1)
    l[0, 5::64] = rng.standard_normal(16)            # all of one lane's
    l[1, 5::64] = rng.standard_normal(16)
    l[1, 6::64] = rng.standard_normal(16)
    l[2, :20] = rng.standard_normal(20)
    l[3, [0, 1023]] = [1.0, 2.0]
    for bias in (None, rng.standard_normal(1024) * 0.1):
        for score in SCORE:
            check_select(up(l), 16, score, bias=bias)
            check_select(up(l), 32, score, bias=bias, num_groups=2, group_limit=1, group_top=2)


@pytest.mark.parametrize("E,k", [(1024, 32), (896, 32), (520, 30), (128, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_select_where_the_best_share_lanes(E, k, score):
    """Experts above all others sit 64 apart, several to a lane, and more than 64 experts lie above the
    k-th of the lanes' best."""
    rng = np.random.default_rng(E)
    l = rng.standard_normal((5, E)).astype(np.float32)
    for t, lanes in enumerate((k - 1, k - 2, 12, 8, 20)):
        e = np.arange(E)
        l[t, e % 64 < lanes] += 6.0
    l[4] = l[4].round(1)   # many equal ones
    for dtype in (F32, BF):
        check_select(up(l).to(dtype), k, score)
        check_select(up(l).to(dtype), k, score, bias=rng.standard_normal(E) * 0.01)
        check_select(up(l).to(dtype), k, score, bias=rng.choice([0.0, INF, -INF], E, p=[0.5, 0.3, 0.2]))
    check_select(up(l), k // 2, score, bias=rng.standard_normal(E) * 0.01, num_groups=2, group_limit=1, group_top=2)


def test_select_keeps_scores_that_underflow():
    """Renormalised weights of experts that only the bias selects: their softmax is below
    fp32's range, the ratio is not."""
    l = np.zeros((1, 10), np.float32)
    l[0, :4] = [-200.0, -201.0, -202.5, 10.0]
    bias = np.zeros(10)
    bias[:3] = 5.0
    for score in ("softmax", "sigmoid"):
        ids, w = check_select(up(l), 3, score, bias=bias, renormalize=True)
        e = np.exp([0.0, -1.0, -2.5])
        assert ids.tolist() == [[0, 1, 2]]
        np.testing.assert_allclose(f64(w)[0], e / e.sum(), rtol=450 * U)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_select_rows_of_a_wider_matrix(dtype):
    """Rows with a stride, from an address that only their type aligns; the rest is NaN."""
    rng = np.random.default_rng(11)
    l = logits_of(rng, 13, 70, dtype)
    wide = torch.full((13, 91), NAN, dtype=dtype, device=dev())
    wide[:, 3:73] = l
    for bias in (None, rng.standard_normal(70)):
        a, b = check_select(l, 5, bias=bias), check_select(wide[:, 3:73], 5, bias=bias)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    dw = up(rng.standard_normal((13, 5)).astype(np.float32))
    for kw in (dict(renormalize=False), {}):
        assert torch.equal(moe.router_select_backward(dw, l, a[0], **kw),
                           moe.router_select_backward(dw, wide[:, 3:73], a[0], **kw))


def test_select_writes_its_rows_alone():
    l = logits_of(np.random.default_rng(1), 9, 24, F32)
    ids = torch.full((11, 4), 77, dtype=I32, device=dev())
    w = torch.full((11, 4), 7.0, device=dev())
    got = moe.router_select(l, 4, ids=ids[1:10], weights=w[1:10])
    assert got[0].data_ptr() == ids[1:10].data_ptr()
    assert (ids[[0, 10]] == 77).all() and (w[[0, 10]] == 7).all() and (ids[1:10] < 24).all()
    assert moe.router_select(l[:0], 4)[0].shape == (0, 4)


def test_select_of_many_tokens():
    """More rows than the grid of one turn holds, against torch on the same ids rule."""
    g = torch.Generator(device=dev()).manual_seed(2)
    l = torch.randn((70001, 40), device=dev(), generator=g)
    ids, w = moe.router_select(l, 6, renormalize=False)
    v, i = l.sort(dim=1, descending=True, stable=True)
    assert torch.equal(ids.long(), i[:, :6])
    want = torch.softmax(l.double(), dim=1).gather(1, i[:, :6])
    assert ((w.double() - want).abs() <= 60 * U * want).all()


def check_select_backward(logits, ids, dw, score, renormalize, scale=1.0):
    got = moe.router_select_backward(dw, logits, ids, score=SCORE[score], renormalize=renormalize, scale=scale)
    assert got.dtype == logits.dtype
    l, i, d = f64(logits), ids.cpu().numpy(), f64(dw)
    want = oracle.router_select_backward(np.nan_to_num(d), l, i, score, renormalize, scale)
    # |dl| is a product of a score and a difference of sums of g and p g: each as in check_select, over k
    # slots; the terms' sizes are those of the differences taken apart
    E = l.shape[1]
    size = np.zeros_like(want)
    for t in range(len(l)):
        live = [s for s in range(i.shape[1]) if 0 <= i[t, s] < E and l[t, i[t, s]] > -np.inf]
        g = np.abs(scale * np.nan_to_num(d[t]))
        s = oracle.scores(l[t], score)
        p = oracle.selected_weights(l[t], i[t], score, renormalize, 1.0)
        mean = sum(p[a] * g[a] for a in live)
        if score == "softmax" and not renormalize:
            size[t] += s * mean
        for a in live:
            size[t, i[t, a]] += p[a] * (g[a] + mean)
    tol = (4 * spread(l) + 120) * U * size + half_step(got) * np.abs(want) + 2.0 ** -125
    assert (np.abs(f64(got) - want) <= tol).all(), np.abs(f64(got) - want).max()
    return got


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 8, 2), (4, 63, 32), (7, 65, 8), (3, 200, 9), (5, 384, 8), (3, 896, 16),
                                   (2, 1024, 32), (301, 8, 2)])
def test_select_backward(T, E, k, score, renormalize, dtype):
    rng = np.random.default_rng(E + 3 * k)
    l = logits_of(rng, T, E, dtype)
    ids, _ = moe.router_select(l, k, score=SCORE[score])
    check_select_backward(l, ids, up(rng.standard_normal((T, k)).astype(np.float32)), score, renormalize, 2.5)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_select_backward_of_any_ids(score, renormalize, dtype):
    """Masked rows and logits, ids of no expert with NaN gradients, ids given twice, extremes."""
    rng = np.random.default_rng(5)
    l = rng.standard_normal((9, 30)).astype(np.float32)
    ids = np.stack([rng.permutation(30)[:6] for _ in range(9)]).astype(np.int32)
    dw = rng.standard_normal((9, 6)).astype(np.float32)
    l[0] = -INF
    l[1, ids[1, 2]] = NAN
    dw[1, 2] = NAN
    ids[2, [0, 4]] = [-1, 30]
    dw[2, [0, 4]] = [NAN, INF]
    ids[3] = [5, 5, 5, 7, 7, 9]
    ids[4] = -1
    dw[4] = NAN
    l[5] = -200.0 + l[5]
    l[6, ids[6, 0]] = torch.finfo(BF).max
    l[7, ids[7, 1]] = torch.finfo(BF).min
    ids[8] = [-2 ** 31, 2 ** 31 - 1, 1024, 63, 29, 0]
    l[0, 0] = -INF
    check_select_backward(up(l).to(dtype), up(ids), up(dw), score, renormalize)


def test_select_backward_against_differences():
    """Central differences of the entry's own weights, step 2^-6: off by the third derivative
    (below 1) times h^2 / 6, and by the two weights' errors over 2 h: 60 u each (check_select's bound
    for logits within 5 of each other), for weights of at most 1."""
    rng = np.random.default_rng(8)
    l = np.round(rng.standard_normal((6, 12)) * 64) / 64
    dw = rng.standard_normal((6, 4)).astype(np.float32)
    h = 2.0 ** -6
    for score in SCORE:
        for renormalize in (True, False):
            kw = dict(score=SCORE[score], renormalize=renormalize)
            ids = moe.router_select(up(l.astype(np.float32)), 4, **kw)[0]
            got = f64(moe.router_select_backward(up(dw), up(l.astype(np.float32)), ids, **kw))
            for e in range(12):
                f = []
                for step in (h, -h):
                    x = l.copy()
                    x[:, e] += step
                    # weights at these ids, by the entry itself with every other expert switched off
                    w = np.zeros((6, 4))
                    for t in range(6):
                        i = ids[t].cpu().numpy()
                        off = np.full(12, -INF)
                        off[i] = 0.0
                        a, b = moe.router_select(up(x[t:t + 1].astype(np.float32)), 4, bias=up(off.astype(np.float32)), **kw)
                        order = {int(v): float(q) for v, q in zip(a[0].tolist(), b[0].tolist())}
                        w[t] = [order[int(v)] for v in i]
                    f.append((w * dw).sum(1))
                err = np.abs((f[0] - f[1]) / (2 * h) - got[:, e])
                assert (err <= np.abs(dw).sum(1) * (h * h / 6 + 60 * U / h)).all(), (score, renormalize, e, err.max())


# ------------------------------------------------------------------ product
def mx(rng, n, k, low=124, high=131):
    return (rng.integers(0, 256, (n, k // 2), dtype=np.uint8), rng.integers(low, high, (n, k // 32), dtype=np.uint8))


def rounded(v, dtype):
    """Nearest value of the type to fp64 values that fp32 holds exactly."""
    f = np.asarray(v, np.float64).astype(np.float32)
    assert (f.astype(np.float64) == v).all()
    return f.astype(np.float64) if dtype == F32 else oracle.bf16_bits_to_f64(oracle.f32_to_bf16_rne(f))


LINEAR_SIZES = [(1, 1, 32), (1, 16, 64), (2, 17, 96), (16, 16, 128), (17, 33, 160), (1, 4096, 1024), (5, 100, 2048),
                (33, 257, 288), (64, 64, 512), (65, 130, 544), (128, 128, 256), (130, 250, 1056), (256, 256, 768),
                (257, 511, 800), (300, 1000, 2048), (513, 264, 4096), (700, 300, 96), (1, 129, 4128), (37, 384, 1376),
                (3, 7168, 2048), (1, 300, 65536), (2000, 1201, 352), (4097, 40, 64),
                # fewer than four scales in all, and rows of x and W that end inside every kind of workgroup
                (3, 1, 96), (70, 3, 32), (5, 2, 32), (4, 4090, 160), (5, 70, 224), (16, 5001, 544), (13, 9001, 416),
                (33, 4090, 160), (50, 7100, 672), (100, 8100, 96), (4, 130, 20000), (9, 66, 20000), (40, 66, 20000),
                (2049, 6100, 96), (1111, 5002, 160)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,n,k", LINEAR_SIZES)
def test_linear_is_exact_on_integers(m, n, k, dtype):
    """x of integers up to 3, scales 2^-1 .. 2^1: multiples of 1/4, sums below 36 k."""
    rng = np.random.default_rng(m + n + k)
    x = rng.integers(-3, 4, (m, k)).astype(np.float32)
    codes, scales = mx(rng, n, k, 126, 129)
    got = moe.mxfp4_linear(up(x).to(BF), up(codes), up(scales), dtype=dtype)
    want = torch.mm(up(x).double(), up(oracle.mxfp4_values(codes, scales)).t().contiguous()).cpu().numpy()
    np.testing.assert_array_equal(f64(got), rounded(want, dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,n,k", [(1, 32, 64), (1, 256, 7168), (7, 130, 2048), (16, 34, 96), (37, 200, 1024), (70, 514, 288),
                                   (300, 258, 640), (1030, 80, 512), (2050, 1154, 160), (4, 2, 32),
                                   (2, 2, 32), (3, 4106, 352), (11, 1030, 224), (16, 5010, 544), (9, 9002, 96), (31, 4118, 96),
                                   (50, 7102, 160), (100, 8110, 96), (2100, 6014, 96), (6, 26, 20000)])
@pytest.mark.parametrize("gate", [False, True])
def test_linear_of_real_values(m, n, k, gate, dtype):
    rng = np.random.default_rng(m * n + k)
    x = up(rng.standard_normal((m, k)).astype(np.float32)).to(BF)
    middle = 127 - int(np.log2(2.9 * np.sqrt(k)))
    codes, scales = mx(rng, n, k, middle - 2, middle + 2)
    got = moe.mxfp4_linear(x, up(codes), up(scales), gate=gate, dtype=dtype)
    w = oracle.mxfp4_values(codes, scales)
    y, size = f64(x) @ w.T, np.abs(f64(x)) @ np.abs(w).T
    dy = k * 2 * U * size       # the MFMA's additions may truncate: a whole step each
    if gate:
        g, u = np.split(y, 2, axis=1)
        dg, du = np.split(dy, 2, axis=1)
        s = g / (1 + np.exp(-g))
        # |silu'| < 1.1; the exponential, the quotient and the product add (|g| + 6) u
        dy = 1.1 * dg * (np.abs(u) + du) + (np.abs(s) + 1.1 * dg) * du + (np.abs(g) + 6) * U * np.abs(s * u)
        y = s * u
        np.testing.assert_allclose(y, oracle.mxfp4_linear(f64(x), codes, scales, gate=True), rtol=1e-9, atol=1e-12)
    tol = dy + half_step(got) * (np.abs(y) + dy)
    assert (np.abs(f64(got) - y) <= tol).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m", [4, 40, 70000, 100000])
def test_linear_gate_far_below_zero(m, dtype):
    """Gates whose exp(-g) passes fp32's range and up to it, times values that bring the product back into
    it. W's rows have one unit weight each, so g and u are x's first two columns, exactly."""
    g = [-89.0, -100.0, -88.5, -103.0, -104.0, -85.0, -87.5, -90.0, -95.0, -110.0, -120.0, -150.0, -176.0,
         -63.75, -64.0, -64.5, -20.0, -1.0, -0.0, 0.0, 1.0, 30.0, 88.0, 89.0, 200.0, 1e30, -1e30]
    u = [-2.0 ** 127, 2.0 ** 100, 2.0 ** 60, -3.0, 1.0]
    pairs = np.array([(a, b) for a in g for b in u if a < 0 or abs(a * b) < 2.0 ** 127])
    x = np.zeros((m, 32), np.float32)
    x[:, :2] = pairs[np.arange(m) % len(pairs)]
    codes = np.zeros((8, 16), np.uint8)
    codes[:4, 0], codes[4:, 0] = 0x02, 0x20        # 1 in column 0 of w1's rows, in column 1 of w3's
    xb = up(x).to(BF)
    got = moe.mxfp4_linear(xb, up(codes), up(np.full((8, 1), 127, np.uint8)), gate=True, dtype=dtype)
    a, b = f64(xb)[:, 0], f64(xb)[:, 1]
    e = np.exp(-np.abs(a))
    want = (a * np.where(a < 0, e, 1.0) / (1.0 + e) * b)[:, None]
    # two exponentials of g / 2, 2 u and their arguments' |g| / 2 u each, three products; below g = -174 the
    # exponential is subnormal: twice 2^-150 off, times |g u exp(g / 2)| < 2^8; bf16's own subnormals: 2^-134
    tol = (np.abs(a) + 7)[:, None] * U * np.abs(want) + 2.0 ** -141
    assert (np.abs(f64(got) - want) <= tol + half_step(got) * (np.abs(want) + tol) + (2.0 ** -134 if dtype == BF else 0)).all()


def test_linear_takes_every_scale_byte():
    """Weights 2^-128 .. 6 2^127 and NaN, exact where the product is: one column a byte."""
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(16, 16), (16, 1))   # every code pair in each block of 16 rows
    scales = np.arange(256, dtype=np.uint8).reshape(256, 1)
    x = np.zeros((3, 32), np.float32)
    x[0, 5] = 1.0
    x[1, 10] = 2.0 ** 100
    x[2, 31] = 2.0 ** -20
    for dtype in (BF, F32):
        got = f64(moe.mxfp4_linear(up(x).to(BF), up(codes), up(scales), dtype=dtype))
        with np.errstate(invalid="ignore", over="ignore"):
            w = oracle.mxfp4_values(codes, scales)
            w = np.where(np.abs(w) >= 2.0 ** 128, np.copysign(np.inf, w), w)
            for r, c in ((0, 5), (1, 10), (2, 31)):
                v = x[r, c].astype(np.float64) * w[:, c]
                v = np.where(np.abs(v) >= 2.0 ** 128, np.copysign(np.inf, v), v)
                # an infinite weight times the other zeros of x is NaN
                bad = np.isnan(w).any(1) | np.isinf(np.delete(w, c, axis=1)).any(1)
                np.testing.assert_array_equal(np.isnan(got[r]), bad | np.isnan(v))
                ok = ~(bad | np.isnan(v))
                if r == 2:   # results below 2^-126 of fp32: at most two bits, exact down to 2^-148
                    ok &= np.abs(v) >= 2.0 ** -126
                np.testing.assert_array_equal(got[r][ok], v[ok])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m", [3, 16, 40, 128, 200, 300, 1000, 8192])
def test_linear_takes_every_scale_byte_beside_others(m, dtype):
    """Every byte as the scale of each block of a row, any other bytes beside it (none of NaN or infinite
    weights, which x's zeros would turn to NaN); x is one value in one block, so products are exact. m reaches
    the streaming kernel's shapes and both tile shapes."""
    blocks = 7                                     # a dword of scales and three bytes of the next
    rng = np.random.default_rng(31)
    n, k = 256 * blocks, 32 * blocks
    scales = rng.choice([0, 1, 2, 3, 63, 64, 126, 127, 128, 129, 191, 250, 251, 252], (n, blocks)).astype(np.uint8)
    at = np.arange(n) // 256                       # the block that a row's byte is tried in
    scales[np.arange(n), at] = np.arange(n) % 256
    codes = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
    row = np.arange(m)
    col = 32 * (row % blocks) + (row // blocks * 5) % 32
    value = np.where(row % 3 == 2, 2.0 ** 100, 1.0) * np.where(row % 2, -1.0, 1.0)
    x = np.zeros((m, k), np.float32)
    x[row, col] = value
    got = moe.mxfp4_linear(up(x).to(BF), up(codes), up(scales), dtype=dtype)
    with np.errstate(over="ignore"):
        w = oracle.mxfp4_values(codes, scales)
    w = np.where(np.abs(w) >= 2.0 ** 128, np.copysign(np.inf, w), w)
    w = up(w)
    want = w[:, up(col)].t() * up(value).unsqueeze(1)
    want = torch.where(want.abs() >= 2.0 ** 128, torch.copysign(torch.full_like(want, INF), want), want)
    # an infinite weight times another zero of x is NaN
    nan, inf = torch.isnan(w).any(1), torch.isinf(w)
    bad = nan | (inf.sum(1).unsqueeze(0) - inf[:, up(col)].t().int() > 0)
    assert torch.equal(torch.isnan(got), bad) and 0 < int(bad.sum()) < bad.numel() // 50
    assert torch.equal(got.double()[~bad], want[~bad])


@pytest.mark.parametrize("m", [1, 20, 200, 2000])
def test_linear_rows_of_a_wider_matrix(m):
    rng = np.random.default_rng(m)
    x = up(rng.standard_normal((m, 160)).astype(np.float32)).to(BF)
    codes, scales = map(up, mx(rng, 300, 160))
    wide = torch.full((m, 160 + 24), NAN, dtype=BF, device=dev())
    wide[:, 8:168] = x
    out = torch.full((m + 2, 300), 5.0, dtype=BF, device=dev())
    got = moe.mxfp4_linear(wide[:, 8:168], codes, scales)
    assert torch.equal(got, moe.mxfp4_linear(x, codes, scales))
    # a contiguous range of a larger output; the rows around it stay
    if m % 2 == 0:
        moe.mxfp4_linear(x, codes, scales, out=out[2:])
        assert torch.equal(out[2:], got) and (out[:2] == 5).all()


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("m", [1, 3, 16, 17, 40, 100, 300, 1100, 9000])
def test_linear_row_does_not_depend_on_other_rows_values(m, gate):
    """NaN and infinite rows next to it change no row's bits."""
    rng = np.random.default_rng(m)
    x = up(rng.standard_normal((m, 288)).astype(np.float32)).to(BF)
    codes, scales = map(up, mx(rng, 290, 288))
    a = moe.mxfp4_linear(x, codes, scales, gate=gate)
    keep = m // 2
    y = torch.full_like(x, NAN)
    y[::2] = INF
    y[keep] = x[keep]
    b = moe.mxfp4_linear(y, codes, scales, gate=gate)
    assert torch.equal(a[keep], b[keep])


def test_linear_of_nothing():
    e = lambda *s, dtype=BF: torch.empty(s, dtype=dtype, device=dev())
    u8 = torch.uint8
    assert moe.mxfp4_linear(e(0, 64), e(5, 32, dtype=u8), e(5, 2, dtype=u8)).shape == (0, 5)
    assert moe.mxfp4_linear(e(3, 64), e(0, 32, dtype=u8), e(0, 2, dtype=u8), gate=True).shape == (3, 0)


def test_linear_beyond_32_bit_offsets():
    """x and out of more than 2^31 elements, and a matrix of more than 2^32 weights."""
    g = torch.Generator(device=dev()).manual_seed(1)
    m, k, n = 300000, 8192, 7200      # 2.46e9 elements of x, 2.16e9 of out
    x = torch.zeros((m, k), dtype=BF, device=dev())
    x[-3:] = torch.randint(-2, 3, (3, k), device=dev(), generator=g).to(BF)
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device=dev(), generator=g)
    scales = torch.full((n, k // 32), 127, dtype=torch.uint8, device=dev())
    out = moe.mxfp4_linear(x, codes, scales)
    assert torch.equal(out[-3:], moe.mxfp4_linear(x[-3:].clone(), codes, scales)) and not out[:-3].any()
    assert out[-3:].any()
    del x, out, codes, scales
    n, k = 1 << 17, 32768 + 64        # 2^32 weights and more, 2.1 GiB of codes
    codes = torch.zeros((n, k // 2), dtype=torch.uint8, device=dev())
    scales = torch.full((n, k // 32), 127, dtype=torch.uint8, device=dev())
    codes[-2:] = torch.randint(0, 256, (2, k // 2), dtype=torch.uint8, device=dev(), generator=g)
    x = torch.randint(-2, 3, (3, k), device=dev(), generator=g).to(BF)
    out = moe.mxfp4_linear(x, codes, scales, dtype=F32)
    want = moe.mxfp4_linear(x, codes[-2:].clone(), scales[-2:].clone(), dtype=F32)
    assert torch.equal(out[:, -2:], want) and want.any() and not out[:, :-2].any()


def test_linear_gated_halves_far_apart():
    """w3 starts 2 GiB behind w1."""
    g = torch.Generator(device=dev()).manual_seed(2)
    n, k = 1 << 18, 32768
    codes = torch.zeros((n, k // 2), dtype=torch.uint8, device=dev())
    scales = torch.full((n, k // 32), 121, dtype=torch.uint8, device=dev())
    rows = [5, n // 2 - 1, n // 2 + 5, n - 1]
    codes[rows] = torch.randint(0, 256, (4, k // 2), dtype=torch.uint8, device=dev(), generator=g)
    for m in (1, 40):
        x = torch.randint(-2, 3, (m, k), device=dev(), generator=g).to(BF)   # sums are exact in any order
        out = moe.mxfp4_linear(x, codes, scales, gate=True, dtype=F32)
        want = moe.mxfp4_linear(x, codes[rows].clone(), scales[:4].clone(), gate=True, dtype=F32)
        assert torch.equal(out[:, [5, n // 2 - 1]], want) and want.any()
        out[:, [5, n // 2 - 1]] = 0
        assert not out.any()


def test_linear_gated_halves_at_the_border_of_32_bit_offsets():
    """w3 starts a few rows less than 2 GiB behind w1: the last size whose rows of w3 the streaming kernel
    reaches from w1's (131054), the first that it does not and the last below 2 GiB."""
    g = torch.Generator(device=dev()).manual_seed(3)
    k = 65536
    codes = torch.zeros((131070, k // 2), dtype=torch.uint8, device=dev())
    scales = torch.full((131070, k // 32), 121, dtype=torch.uint8, device=dev())
    for n in (131054, 131056, 131070):
        half = n // 2
        cols = [*range(16), 32767, *range(half - 9, half)]       # every row of the first and the last workgroups
        rows = cols + [half + c for c in cols]
        codes[rows] = torch.randint(0, 256, (len(rows), k // 2), dtype=torch.uint8, device=dev(), generator=g)
        for m in (1, 3, 16):
            x = torch.randint(-2, 3, (m, k), device=dev(), generator=g).to(BF)   # sums are exact in any order
            out = moe.mxfp4_linear(x, codes[:n], scales[:n], gate=True, dtype=F32)
            want = moe.mxfp4_linear(x, codes[rows].clone(), scales[:len(rows)].clone(), gate=True, dtype=F32)
            assert want.any(0).all() and torch.equal(out[:, cols], want), (n, m)
            out[:, cols] = 0
            assert not out.any(), (n, m)
        codes[rows] = 0


@pytest.mark.parametrize("m", [3, 40, 300])
def test_linear_rows_as_far_apart_as_they_may_be(m):
    rng = np.random.default_rng(m)
    x = up(rng.standard_normal((m, 352)).astype(np.float32)).to(BF)
    codes, scales = map(up, mx(rng, 200, 352))
    wide = torch.empty((m, 1 << 20), dtype=BF, device=dev())[:, :352]
    wide.copy_(x)
    assert torch.equal(moe.mxfp4_linear(wide, codes, scales), moe.mxfp4_linear(x, codes, scales))


# ------------------------------------------------------------------ combine
def routes(rng, T, k, experts, resident):
    """(rowpos [T, k], perm [T k], valid) of random ids, as the layer's route stage sorts them."""
    ids = rng.integers(0, experts, T * k)
    order = np.argsort(np.where(ids < resident, ids, experts), kind="stable")
    n = int((ids < resident).sum())
    perm, rowpos = np.full(T * k, -7, np.int32), np.full(T * k, -1, np.int32)
    perm[:n] = order[:n]
    rowpos[order[:n]] = np.arange(n)
    return rowpos.reshape(T, k), perm, n


COMBINE_SIZES = [(1, 1, 8), (2, 3, 16), (5, 2, 72), (3, 8, 512), (7, 16, 520), (4, 9, 2048), (130, 8, 1024), (2, 32, 7168),
                 (3, 5, 8200), (1, 2, 65536), (33, 17, 4104)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,k,H", COMBINE_SIZES)
def test_combine(T, k, H, dtype):
    """Integer rows and weights: exact in any order."""
    rng = np.random.default_rng(T + k + H)
    rowpos, perm, n = routes(rng, T, k, 8, 6)
    y = rng.integers(-8, 9, (T * k, H)).astype(np.float32)
    y[n:] = NAN        # rows that no route has are not read
    w = rng.integers(-3, 4, (T, k)).astype(np.float32)
    w[rowpos < 0] = NAN
    for weights in (w, None):
        got = moe.expert_combine(up(y).to(BF), up(rowpos), None if weights is None else up(weights), dtype=dtype)
        want = oracle.expert_combine(y, rowpos, weights)
        np.testing.assert_array_equal(f64(got), rounded(want, dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,k,H", [(6, 8, 264), (9, 16, 1024), (40, 2, 4096)])
def test_combine_of_real_values(T, k, H, dtype):
    rng = np.random.default_rng(H)
    rowpos, perm, n = routes(rng, T, k, 5, 5)
    y = up(rng.standard_normal((T * k, H)).astype(np.float32)).to(BF)
    w = up(rng.random((T, k)).astype(np.float32))
    got = moe.expert_combine(y, up(rowpos), w, dtype=dtype)
    want = oracle.expert_combine(f64(y), rowpos, f64(w))
    size = oracle.expert_combine(np.abs(f64(y)), rowpos, f64(w))
    tol = k * U * size     # one rounding a multiply-add
    assert (np.abs(f64(got) - want) <= tol + half_step(got) * (np.abs(want) + tol)).all()


def test_combine_of_any_rows():
    """Rows outside [0, rows), the same row for several slots, no row at all, no rows there."""
    rng = np.random.default_rng(2)
    y = rng.integers(-8, 9, (5, 40)).astype(np.float32)
    rowpos = np.array([[0, 0, 0], [5, -2 ** 31, 2 ** 31 - 1], [4, 5, 4], [-1, -1, -1], [1, 2, 3]], np.int32)
    w = np.array([[1, 2, 3], [NAN, NAN, NAN], [2, INF, 1], [NAN, 0, INF], [1, -1, 2]], np.float32)
    got = moe.expert_combine(up(y).to(BF), up(rowpos), up(w), dtype=F32)
    np.testing.assert_array_equal(f64(got), oracle.expert_combine(y, rowpos, w))
    none = moe.expert_combine(up(y[:0]).to(BF), up(rowpos), up(w))
    assert none.shape == (5, 40) and not none.any()
    assert moe.expert_combine(up(y).to(BF), up(rowpos[:0]), up(w[:0])).shape == (0, 40)


def test_combine_rows_of_wider_matrices():
    rng = np.random.default_rng(4)
    rowpos, perm, n = routes(rng, 11, 4, 6, 5)
    y = up(rng.integers(-8, 9, (44, 136)).astype(np.float32)).to(BF)
    w = up(rng.random((11, 4)).astype(np.float32))
    wide = torch.full((44, 200), NAN, dtype=BF, device=dev())
    wide[:, 16:152] = y
    a, b = (moe.expert_combine(t, up(rowpos), w) for t in (y, wide[:, 16:152]))
    assert torch.equal(a, b)
    for dtype in (BF, F32):
        dout = up(rng.standard_normal((11, 136)).astype(np.float32)).to(dtype)
        wide_d = torch.full((11, 152), NAN, dtype=dtype, device=dev())
        wide_d[:, 8:144] = dout
        dy = [torch.zeros((44, 136), dtype=BF, device=dev()) for _ in range(2)]
        a = moe.expert_combine_backward(dout, y, up(rowpos), up(perm), w, dy=dy[0])
        b = moe.expert_combine_backward(wide_d[:, 8:144], wide[:, 16:152], up(rowpos), up(perm), w, dy=dy[1])
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,k,H", COMBINE_SIZES)
def test_combine_backward(T, k, H, dtype):
    """Integers: dy is the nearest bf16 of exact products, dweights exact sums."""
    rng = np.random.default_rng(T * k + H)
    rowpos, perm, n = routes(rng, T, k, 8, 6)
    y = rng.integers(-4, 5, (T * k, H)).astype(np.float32)
    y[n:] = NAN
    w = rng.integers(-60, 61, (T, k)).astype(np.float32)
    w[rowpos < 0] = NAN
    dout = rng.integers(-9, 10, (T, H)).astype(np.float32)
    before = torch.full((T * k, H), 3.0, dtype=BF, device=dev())
    for weights in (w, None):
        dy = before.clone()
        t = None if weights is None else up(weights)
        got = moe.expert_combine_backward(up(dout).to(dtype), up(y).to(BF), up(rowpos), up(perm), t, dy=dy)
        want = oracle.expert_combine_backward(dout, y, rowpos, perm, weights, f64(before))
        assert got[0] is dy
        np.testing.assert_array_equal(f64(dy), rounded(want[0], BF))   # rows without a route stay 3
        np.testing.assert_array_equal(f64(got[1]), want[1])
        # each gradient alone
        only = moe.expert_combine_backward(up(dout).to(dtype), None, up(rowpos), up(perm), t, dy=before.clone(), need_dw=False)
        assert only[1] is None and torch.equal(only[0], dy)
        only = moe.expert_combine_backward(up(dout).to(dtype), up(y).to(BF), up(rowpos), None, t, need_dy=False)
        assert only[0] is None and torch.equal(only[1], got[1])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,k,H", [(6, 8, 264), (9, 16, 1024), (40, 2, 7168), (2, 1, 8232)])
def test_combine_backward_of_real_values(T, k, H, dtype):
    rng = np.random.default_rng(H + 1)
    rowpos, perm, n = routes(rng, T, k, 5, 5)
    y = up(rng.standard_normal((T * k, H)).astype(np.float32)).to(BF)
    w = up(rng.random((T, k)).astype(np.float32))
    dout = up(rng.standard_normal((T, H)).astype(np.float32)).to(dtype)
    dy, dw = moe.expert_combine_backward(dout, y, up(rowpos), up(perm), w)
    want_dy, want_dw = oracle.expert_combine_backward(f64(dout), f64(y), rowpos, perm, f64(w), np.zeros((T * k, H)))
    # a product in fp32, then in bf16
    assert (np.abs(f64(dy) - want_dy) <= (2.0 ** -8 + 2 * U) * np.abs(want_dy)).all()
    size = oracle.expert_combine_backward(np.abs(f64(dout)), np.abs(f64(y)), rowpos, perm, f64(w), np.zeros((T * k, H)))[1]
    assert (np.abs(f64(dw) - want_dw) <= H * U * size).all()


def test_combine_backward_of_any_indexes():
    """A row that several slots name gets the gradient of the one that perm names; rowpos outside the
    rows, perm that names no route or another one: nothing is written there."""
    rng = np.random.default_rng(6)
    y = rng.integers(-4, 5, (6, 24)).astype(np.float32)
    dout = rng.integers(-9, 10, (4, 24)).astype(np.float32)
    rowpos = np.array([[0, 0], [0, 3], [6, -2 ** 31], [5, 2 ** 31 - 1]], np.int32)
    perm = np.array([2, 0, -7, 2 ** 31 - 1, -2 ** 31, 6], np.int32)   # rows 0 and 5 belong to routes 2 and 6
    w = np.array([[1, 2], [3, 4], [NAN, NAN], [5, NAN]], np.float32)
    dy = torch.full((6, 24), 7.0, dtype=BF, device=dev())
    got = moe.expert_combine_backward(up(dout), up(y).to(BF), up(rowpos), up(perm), up(w), dy=dy)
    want = oracle.expert_combine_backward(dout, y, rowpos, perm, w, np.full((6, 24), 7.0))
    np.testing.assert_array_equal(f64(dy), want[0])
    np.testing.assert_array_equal(f64(got[1]), want[1])
    assert (dy[[1, 2, 3, 4]] == 7).all()
    none = moe.expert_combine_backward(up(dout), up(y[:0]).to(BF), up(rowpos), up(perm[:0]), up(w))
    assert none[0].shape == (0, 24) and not none[1].any()
    none = moe.expert_combine_backward(up(dout[:0]), up(y).to(BF), up(rowpos[:0]), up(perm), up(w[:0]), dy=dy.clone())
    assert torch.equal(none[0], dy) and none[1].shape == (0, 2)


def test_combine_backward_keeps_nan_where_it_is():
    """A NaN of dout reaches its own column of dy and its token's dweights alone."""
    rng = np.random.default_rng(9)
    rowpos, perm, n = routes(rng, 5, 3, 4, 4)
    y = up(rng.standard_normal((15, 64)).astype(np.float32)).to(BF)
    dout = up(rng.standard_normal((5, 64)).astype(np.float32))
    dout[2, 10] = NAN
    dy, dw = moe.expert_combine_backward(dout, y, up(rowpos), up(perm))
    rows = torch.isnan(dy).nonzero()
    assert sorted(map(tuple, rows.tolist())) == sorted((int(r), 10) for r in rowpos[2])
    assert torch.isnan(dw).nonzero().tolist() == [[2, 0], [2, 1], [2, 2]]


def test_combine_beyond_32_bit_offsets():
    """y and dy of more than 2^31 elements."""
    rows, H = 280000, 8192
    y = torch.zeros((rows, H), dtype=BF, device=dev())
    y[-2] = 2.0
    y[5] = 1.0
    rowpos = torch.tensor([[5, rows - 2], [rows - 1, -1]], dtype=I32, device=dev())
    w = torch.tensor([[1.0, 3.0], [1.0, 1.0]], device=dev())
    out = moe.expert_combine(y, rowpos, w)
    assert (out[0] == 7).all() and (out[1] == 0).all()
    perm = torch.full((rows,), -7, dtype=I32, device=dev())
    perm[5], perm[rows - 2], perm[rows - 1] = 0, 1, 2
    dout = torch.ones((2, H), device=dev())
    dout[1] = 4.0
    keep = torch.zeros((rows, H), dtype=BF, device=dev())
    dy, dw = moe.expert_combine_backward(dout, y, rowpos, perm, w, dy=keep)
    assert (dy[5] == 1).all() and (dy[-2] == 3).all() and (dy[-1] == 4).all()
    assert int((dy != 0).any(1).sum()) == 3
    assert dw.tolist() == [[float(H), 2.0 * H], [0.0, 0.0]]


# ------------------------------------------------------------------ the largest sizes
def test_select_of_the_most_tokens():
    """2^24 rows of 8 experts: every row is one of 64, so all results are its own row's."""
    T, k = 1 << 24, 2
    rng = np.random.default_rng(41)
    few = logits_of(rng, 64, 8, F32)
    few[3] = -INF
    l = few.repeat(T // 64, 1)
    ids, w = moe.router_select(l, k, score=moe.MOE_SCORE_SIGMOID)
    want = moe.router_select(few, k, score=moe.MOE_SCORE_SIGMOID)
    check_select(few, k, "sigmoid")
    assert (ids.view(-1, 64, k) == want[0]).all() and (w.view(-1, 64, k) == want[1]).all()
    dw = up(rng.standard_normal((64, k)).astype(np.float32))
    got = moe.router_select_backward(dw.repeat(T // 64, 1), l, ids, score=moe.MOE_SCORE_SIGMOID)
    want = moe.router_select_backward(dw, few, want[0], score=moe.MOE_SCORE_SIGMOID)
    assert (got.view(-1, 64, 8) == want).all()


@pytest.mark.parametrize("m,n,k,gate", [(1 << 19, 18, 64, True), (5, 1 << 19, 96, False), (40, 1 << 19, 32, True),
                                        (1 << 19, 1, 32, False), (300, 514, 65536, True), (16, 48, 65536, False),
                                        (17, 4100, 65536, False)])
def test_linear_at_its_limits(m, n, k, gate):
    """Integer x and scales as in the exact test; sums below 2^24 quarters."""
    rng = np.random.default_rng(43)
    g = torch.Generator(device=dev()).manual_seed(43)
    x = torch.randint(-1, 2, (m, k), device=dev(), generator=g).to(BF)
    codes, scales = mx(rng, n, k, 126, 128)
    got = moe.mxfp4_linear(x, up(codes), up(scales), gate=gate, dtype=F32)
    w = up(oracle.mxfp4_values(codes, scales)).float()
    y = torch.mm(x.float(), w.t().contiguous())     # exact: multiples of 1/4 below 2^20
    if not gate:
        assert torch.equal(got, y)
        return
    y = y.double()
    a, u = y.chunk(2, dim=1)
    want = a * torch.special.expit(a) * u
    # two exponentials' arguments and three operations, as counted for gates far below zero
    assert ((got.double() - want).abs() <= (a.abs() + 7) * U * want.abs() + 2.0 ** -139).all()


def test_combine_of_the_most_tokens_and_slots():
    """2^21 tokens of 32 slots; hidden 8. Slot s of token t is row 32 t + s, or none where t + s is a multiple of 5."""
    T, k, H = 1 << 21, 32, 8
    rows = T * k
    at = torch.arange(rows, dtype=I32, device=dev())
    none = (at // k + at % k) % 5 == 0
    rowpos = at.masked_fill(none, -1).view(T, k)
    perm = at.masked_fill(none, -7)
    y = (at % 7 - 3).to(BF).unsqueeze(1).repeat(1, H)
    y[:, 1:] = y[:, 1:] * torch.arange(1, H, device=dev(), dtype=torch.float32).to(BF)
    out = moe.expert_combine(y, rowpos, dtype=F32)
    want = y.masked_fill(none.unsqueeze(1), 0).view(T, k, H).float().sum(1)
    assert torch.equal(out, want)
    w = (at % 3 + 1).float().view(T, k)
    dout = (torch.arange(T, device=dev()) % 11 - 5).to(BF).unsqueeze(1).repeat(1, H)
    dy, dw = moe.expert_combine_backward(dout, y, rowpos, perm, w, dy=torch.full_like(y, 7.0))
    want = (w.unsqueeze(2) * dout.float().unsqueeze(1)).to(BF).view(rows, H)
    assert torch.equal(dy, want.masked_fill(none.unsqueeze(1), 7.0))
    want = (y.view(T, k, H).float() * dout.float().unsqueeze(1)).sum(2).masked_fill(none.view(T, k), 0)
    assert torch.equal(dw, want)


# ------------------------------------------------------------------ streams, graphs, and all of them together
def some_calls():
    """(callables, each a pass through one entry on inputs of its own, and the inputs to change)."""
    rng = np.random.default_rng(12)
    l = logits_of(rng, 50, 96, F32)
    bias = up(rng.standard_normal(96).astype(np.float32))
    ids = moe.router_select(l, 6)[0]
    dw = up(rng.standard_normal((50, 6)).astype(np.float32))
    x = up(rng.standard_normal((50, 512)).astype(np.float32)).to(BF)
    x1 = x[:1].clone()
    big = up(rng.standard_normal((700, 512)).astype(np.float32)).to(BF)
    codes, scales = map(up, mx(rng, 640, 512))
    rowpos, perm, n = routes(rng, 50, 6, 8, 6)
    rowpos, perm = up(rowpos), up(perm)
    y = up(rng.standard_normal((300, 512)).astype(np.float32)).to(BF)
    dy = torch.zeros((300, 512), dtype=BF, device=dev())
    flat = lambda *t: tuple(t)
    calls = [lambda: flat(*moe.router_select(l, 6, score=1, bias=bias, num_groups=8, group_limit=3, group_top=2)),
             lambda: flat(*moe.router_select(l, 6, renormalize=False)),
             lambda: flat(moe.router_select_backward(dw, l, ids)),
             lambda: flat(moe.router_select_backward(dw, l, ids, renormalize=False)),
             lambda: flat(moe.mxfp4_linear(x, codes, scales, gate=True)),
             lambda: flat(moe.mxfp4_linear(x1, codes, scales)),
             lambda: flat(moe.mxfp4_linear(big, codes, scales)),
             lambda: flat(moe.expert_combine(y, rowpos, dw)),
             lambda: flat(*moe.expert_combine_backward(x, y, rowpos, perm, dw, dy=dy))]
    return calls, (l, x, x1, big, y, dw)


def test_other_stream():
    """Results made on another stream, behind work that delays it, wait for the inputs made there."""
    calls, inputs = some_calls()
    want = [tuple(t.clone() for t in c()) for c in calls]
    originals = [t.clone() for t in inputs]
    for t in inputs:
        t.zero_()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    busy = torch.ones((4096, 4096), dtype=BF, device=dev())
    with torch.cuda.stream(s):
        for _ in range(8):
            busy = busy @ busy * 1e-4
        for t, o in zip(inputs, originals):
            t.copy_(o)
        got = [tuple(t.clone() for t in c()) for c in calls]
    s.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_two_streams_at_once():
    """The same calls on two streams, enqueued in turn, share no memory."""
    calls, _ = some_calls()
    others, _ = some_calls()
    want = [tuple(t.clone() for t in c()) for c in calls]
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        for a, b in zip(calls, others):
            for s, c in zip(streams, (a, b)):
                with torch.cuda.stream(s):
                    got.append(tuple(t.clone() for t in c()))
    torch.cuda.synchronize()
    for i, res in enumerate(got):
        assert all(torch.equal(p, q) for p, q in zip(res, want[i // 2 % len(want)])), i


def test_stream_argument():
    """stream= alone, without a stream context; memory of temporaries stays with that stream."""
    calls, (l, x, x1, big, y, dw) = some_calls()
    want = moe.router_select(l, 6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = moe.router_select(l, 6, stream=s)
    back = moe.router_select_backward(dw, l, got[0], stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(back, moe.router_select_backward(dw, l, want[0]))


def test_graph_replays_match_eager():
    calls, inputs = some_calls()
    originals = [t.clone() for t in inputs]
    for c in calls:
        c()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):      # two graphs of the same calls share nothing but inputs and dy
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = [c() for c in calls]
        graphs.append((g, res))
    for turn in range(3):
        for t, o in zip(inputs, originals):
            t.copy_(o * (0.5 + turn))
        torch.cuda.synchronize()
        want = [tuple(t.clone() for t in c()) for c in calls]
        torch.cuda.synchronize()
        for g, res in graphs:
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(res, want):
                assert all(torch.equal(p, q) for p, q in zip(a, b)), turn


def test_runs_are_reproducible():
    calls, _ = some_calls()
    first = [tuple(t.clone() for t in c()) for c in calls]
    for _ in range(3):
        for a, c in zip(first, calls):
            assert all(torch.equal(bits(p), bits(q)) for p, q in zip(a, c()))


def plan_of(H, I, E, k, T, rng):
    cfg = moe.Config(H, I, E, k, T)
    w13 = mx(rng, E * 2 * I, H, 120, 124)
    w2 = mx(rng, E * H, I, 120, 124)
    shaped = [up(w13[0].reshape(E, 2 * I, H // 2)), up(w13[1].reshape(E, 2 * I, H // 32)),
              up(w2[0].reshape(E, H, I // 2)), up(w2[1].reshape(E, H, I // 32))]
    return moe.Plan(cfg, *shaped), (w13, w2)


def test_training_step_of_a_routed_projection():
    """Logits to loss and back: router_select, route, gather, grouped_matmul, expert_combine, and every
    gradient, each entry's against the fp64 definition on the values that the step itself made."""
    rng = np.random.default_rng(20)
    T, E, k, H, N = 37, 8, 3, 256, 128
    plan, _ = plan_of(H, 128, E, k, T, rng)
    x = up(rng.standard_normal((T, H)).astype(np.float32)).to(BF)
    w = up((rng.standard_normal((E, N, H)) / 16).astype(np.float32)).to(BF)
    logits = logits_of(rng, T, E, F32)
    logits[5] = -INF                                   # a padded token
    bias = up((rng.standard_normal(E) * 0.1).astype(np.float32))
    rule = dict(score=moe.MOE_SCORE_SIGMOID, scale=1.5)
    ids, wts = moe.router_select(logits, k, bias=bias, num_groups=4, group_limit=2, group_top=2, **rule)
    counts, offsets, perm, rowpos = plan.route(ids)
    rowpos = rowpos.view(T, k)
    n = int(offsets[-1])
    assert n == (T - 1) * k and (rowpos[5] == -1).all()
    rows = moe.expert_combine_backward(x, None, rowpos, perm, need_dw=False, dy=torch.zeros((T * k, H), dtype=BF, device=dev()))[0]
    assert torch.equal(rows[:n], x[perm[:n].long() // k])
    y = moe.grouped_matmul(rows, w, offsets, out=torch.zeros((T * k, N), dtype=BF, device=dev()))
    out = moe.expert_combine(y, rowpos, wts, dtype=F32)
    # loss = sum(c out)
    c = up(rng.standard_normal((T, N)).astype(np.float32))
    dy, dwts = moe.expert_combine_backward(c, y, rowpos, perm, wts, dy=torch.zeros_like(y))
    drows, dw = moe.grouped_matmul_backward(dy, rows, w, offsets, dx=torch.zeros_like(rows))
    dx = moe.expert_combine(drows, rowpos, dtype=F32)
    dlogits = moe.router_select_backward(dwts, logits, ids, **rule)

    # the same step in fp64 by autograd; the ids are the selection's
    lx, lw, ll = (t.double().cpu().requires_grad_() for t in (x, w, logits.nan_to_num(neginf=-50.0)))
    i = ids.cpu().long()
    live = (i >= 0)
    s = torch.sigmoid(ll).gather(1, i.clamp(min=0)) * live
    p = 1.5 * s / s.sum(1, keepdim=True).clamp(min=1e-300)
    per_route = torch.einsum("th,tknh->tkn", lx, lw[i.clamp(min=0)])
    ref = (per_route * p.unsqueeze(-1)).sum(1)
    (ref * c.double().cpu()).sum().backward()
    # y is rounded to bf16 (2^-8), and so are dy and drows: each output is off by that share of its terms
    size = (per_route.abs() * p.unsqueeze(-1)).sum(1).detach().numpy()
    assert (np.abs(f64(out) - ref.detach().numpy()) <= 1.02 * 2.0 ** -8 * size + 1e-6).all()
    terms = lambda a, b: np.abs(a) @ np.abs(b)
    cd = f64(c)
    dw_size, dx_size = np.zeros((E, N, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e = int(i[t, j])
            if e < 0:
                continue
            q = float(p[t, j].detach())
            dw_size[e] += q * np.outer(np.abs(cd[t]), np.abs(f64(x)[t]))
            dx_size[t] += q * terms(cd[t], f64(w)[e])
    assert (np.abs(f64(dw) - lw.grad.numpy()) <= 1.02 * 2.0 ** -8 * dw_size + 1e-6).all()
    assert (np.abs(f64(dx) - lx.grad.numpy()) <= 2.04 * 2.0 ** -8 * dx_size + 1e-6).all()
    # dweights = <c, y>, y rounded; dlogits a combination of them with weights p (|g| + sum p |g|) <= 2 max
    dwt_err = 1.02 * 2.0 ** -8 * (np.abs(cd)[:, None, :] * per_route.abs().detach().numpy()).sum(-1) + 1e-5
    assert (np.abs(f64(dlogits) - ll.grad.numpy()) <= 2 * 1.5 * dwt_err.max(1, keepdims=True) + 1e-5).all()
    assert (dlogits[5] == 0).all() and (out[5] == 0).all() and (dx[5] == 0).all()


def test_serving_step_with_a_shared_expert():
    """router_select feeds the layer's forward; a shared expert's two products run beside it."""
    rng = np.random.default_rng(21)
    T, E, k, H, I = 5, 8, 2, 256, 128
    plan, (w13, w2) = plan_of(H, I, E, k, T, rng)
    x = up(rng.standard_normal((T, H)).astype(np.float32)).to(BF)
    logits = logits_of(rng, T, E, BF)
    ids, wts = moe.router_select(logits, k, score=moe.MOE_SCORE_SIGMOID)
    routed = plan.forward(x, ids, wts)
    case = [a.reshape(s) for a, s in ((w13[0], (E, 2 * I, H // 2)), (w13[1], (E, 2 * I, H // 32)),
                                      (w2[0], (E, H, I // 2)), (w2[1], (E, H, I // 32)))]
    x_bits = x.view(torch.int16).cpu().numpy().view(np.uint16)
    ref = oracle.forward(x_bits, ids.cpu().numpy(), wts.cpu().numpy(), case, E)
    assert oracle.check_rows(f64(routed), ref)["pass"]
    s13, s2 = mx(rng, 2 * I, H, 120, 124), mx(rng, H, I, 120, 124)
    for rows in (x, x[:1]):
        h = moe.mxfp4_linear(rows, *map(up, s13), gate=True)
        shared = moe.mxfp4_linear(h, *map(up, s2), dtype=F32)
        want_h = oracle.mxfp4_linear(f64(rows), *s13, gate=True)
        # fp32 sums of 256 products: 256 2^-23 of their sizes; then half a bf16 step
        w = oracle.mxfp4_values(*s13)
        size = np.abs(f64(rows)) @ np.abs(w).T
        g, u = np.split(f64(rows) @ w.T, 2, axis=1)
        sg, su = np.split(H * 2 * U * size, 2, axis=1)
        tol = 1.1 * sg * (np.abs(u) + su) + (np.abs(g) + 1.1 * sg) * su + (np.abs(g) + 6) * U * np.abs(want_h)
        assert (np.abs(f64(h) - want_h) <= tol + 2.0 ** -8 * (np.abs(want_h) + tol)).all()
        want = oracle.mxfp4_linear(f64(h), *s2)
        size = np.abs(f64(h)) @ np.abs(oracle.mxfp4_values(*s2)).T
        assert (np.abs(f64(shared) - want) <= I * 2 * U * size).all()
