"""The fp64 definitions of the scored router, the product with an MXFP4 matrix
and the experts' combine, pinned by closed forms, torch and differences."""
import numpy as np
import pytest
import torch

import oracle

INF, NAN = np.inf, np.nan


def test_selection_by_hand():
    l = [[1.0, 3.0, 2.0, 3.0, 0.0, -1.0]]
    ids, w = oracle.router_select(l, 3)
    np.testing.assert_array_equal(ids, [[1, 3, 2]])
    e = np.exp([0.0, 0.0, -1.0])
    np.testing.assert_allclose(w[0], e / e.sum(), rtol=1e-15)
    # a bias moves the selection and not the weights
    ids, w = oracle.router_select(l, 2, score="sigmoid", bias=[0, 0, 0, 0, 5.0, -INF], renormalize=False, scale=2.0)
    np.testing.assert_array_equal(ids, [[4, 1]])
    np.testing.assert_allclose(w[0], [1.0, 2.0 / (1 + np.exp(-3.0))], rtol=1e-15)
    # three groups of two: sums of two scores keep (1, 3) and (2, 3); best alone as well, the lower group first
    ids, _ = oracle.router_select(l, 2, num_groups=3, group_limit=1, group_top=2)
    np.testing.assert_array_equal(ids, [[3, 2]])
    ids, _ = oracle.router_select(l, 2, num_groups=3, group_limit=1, group_top=1)
    np.testing.assert_array_equal(ids, [[1, 0]])


def test_selection_of_masked_rows():
    l = [[-INF, NAN, -INF, -INF], [-INF, 2.0, NAN, -INF], [INF, 1.0, INF, NAN]]
    ids, w = oracle.router_select(l, 3)
    np.testing.assert_array_equal(ids, [[-1, -1, -1], [1, -1, -1], [0, 2, 1]])
    np.testing.assert_array_equal(w, [[0, 0, 0], [1, 0, 0], [0.5, 0.5, 0]])
    assert (oracle.router_select_backward(np.full((3, 3), NAN), l, np.full((3, 3), -1)) == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_weights_against_torch(score, renormalize):
    rng = np.random.default_rng(1)
    l = rng.standard_normal((9, 20)) * 3
    ids, w = oracle.router_select(l, 5, score=score, renormalize=renormalize, scale=1.5)
    t = torch.from_numpy(l)
    s = torch.sigmoid(t) if score == "sigmoid" else torch.softmax(t, dim=1)
    top = torch.topk(s, 5, dim=1)
    np.testing.assert_array_equal(ids, top.indices.numpy())
    v = top.values / top.values.sum(1, keepdim=True) if renormalize else top.values
    np.testing.assert_allclose(w, 1.5 * v.numpy(), rtol=1e-14)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_against_differences(score, renormalize):
    """Central differences of step h of a smooth function of size O(1): off by about
    h^2 = 1e-10 and 2^-52 / h = 2e-11."""
    rng = np.random.default_rng(2)
    l = rng.standard_normal((4, 7))
    ids = oracle.router_select(l, 3, score=score)[0]
    ids[1] = [2, 2, 5]       # an id given twice
    ids[2, 1] = -1           # no expert
    l[3, 6] = -INF
    dw = rng.standard_normal((4, 3))
    got = oracle.router_select_backward(dw, l, ids, score, renormalize, 2.0)
    h = 1e-5
    for t in range(4):
        for e in range(7):
            if l[t, e] == -INF:
                assert got[t, e] == 0
                continue
            f = []
            for step in (h, -h):
                x = l[t].copy()
                x[e] += step
                f.append(dw[t] @ oracle.selected_weights(x, ids[t], score, renormalize, 2.0))
            assert abs((f[0] - f[1]) / (2 * h) - got[t, e]) < 2e-9, (t, e)


def test_linear_and_gate():
    rng = np.random.default_rng(3)
    codes, scales = rng.integers(0, 256, (6, 32), dtype=np.uint8), rng.integers(120, 130, (6, 2), dtype=np.uint8)
    x = rng.standard_normal((3, 64))
    w = oracle.mxfp4_values(codes, scales)
    np.testing.assert_allclose(oracle.mxfp4_linear(x, codes, scales), x @ w.T, rtol=1e-15)
    g = torch.from_numpy(x @ w[:3].T)
    want = torch.nn.functional.silu(g).numpy() * (x @ w[3:].T)
    np.testing.assert_allclose(oracle.mxfp4_linear(x, codes, scales, gate=True), want, rtol=1e-12)


def test_combine_and_gradients_against_autograd():
    rng = np.random.default_rng(4)
    ids = rng.integers(-1, 4, (5, 3))
    flat = ids.reshape(-1)
    order = np.argsort(np.where(flat < 0, 9, flat), kind="stable")
    n = int((flat >= 0).sum())
    perm = np.full(15, -7)
    perm[:n] = order[:n]
    rowpos = np.full(15, -1)
    rowpos[order[:n]] = np.arange(n)
    rowpos = rowpos.reshape(5, 3)
    y = torch.from_numpy(rng.standard_normal((15, 8))).requires_grad_()
    w = torch.from_numpy(rng.standard_normal((5, 3))).requires_grad_()
    live = torch.from_numpy(rowpos >= 0)
    out = (y[torch.from_numpy(np.maximum(rowpos, 0))] * (w * live).unsqueeze(-1)).sum(1)
    np.testing.assert_allclose(oracle.expert_combine(y.detach().numpy(), rowpos, w.detach().numpy()),
                               out.detach().numpy(), rtol=1e-14, atol=1e-15)
    dout = rng.standard_normal((5, 8))
    out.backward(torch.from_numpy(dout))
    gy, gw = oracle.expert_combine_backward(dout, y.detach().numpy(), rowpos, perm, w.detach().numpy(), np.zeros((15, 8)))
    np.testing.assert_allclose(gy, y.grad.numpy(), rtol=1e-14)
    np.testing.assert_allclose(gw, w.grad.numpy(), rtol=1e-13, atol=1e-14)
    # weights of 1 gather dout's rows into the experts' order
    rows = oracle.expert_combine_backward(dout, y.detach().numpy(), rowpos, perm, None, np.zeros((15, 8)))[0]
    np.testing.assert_array_equal(rows[:n], dout[perm[:n] // 3])
