"""Measured cases of the scored router, of products with MXFP4 weights and of the experts' combine.

Operators, and the entry points that `run` calls where `own` is true:
  select            router_select: scores, a bias for balance, expert groups, top-k, renormalised weights
  select_backward   router_select_backward: the logits' gradient from the weights'
  linear            mxfp4_linear: bf16 rows times an MXFP4 matrix, plain or with the SiLU gate of w1||w3
  combine           expert_combine: each token's weighted sum of its routes' rows
  combine_backward  expert_combine_backward: gradients of the rows and of the weights

Where `own` is false the same results are computed from elementary torch
operations in fp32, rounded once at the end; the router's selection values are
fp64, because ids change where two of them lie within a rounding of each other.
"""
import math

import numpy as np
import torch

own = False

GROUP = 32                                             # weights per E8M0 scale
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)        # magnitudes of the E2M1 codes 0..7
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SCORES = ("softmax", "sigmoid")
FLOAT_MAX = torch.finfo(torch.float32).max

# Sizes of the layer's own workloads: hidden 7168, intermediate 2048 (a fused
# w1||w3 matrix is [4096, 7168], w2 [7168, 2048]); 384 experts, top-8, or 896
# experts, top-16; 1 to 4096 tokens, here up to four such batches.
MOST_LOGITS = 16384 * 896
MOST_LINEAR = 4096 * 4096 * 7168
MOST_ROUTED = 4096 * 8 * 7168


def listed():
    return [
        # one decoded token: sigmoid scores, a bias, eight groups of which four are kept
        {"name": "select_one_token", "op": "select", "tokens": 1, "pad": 0, "experts": 384, "top_k": 8,
         "score": "sigmoid", "bias": True, "groups": 8, "limit": 4, "group_top": 2, "renormalize": True,
         "scale": 2.5, "dtype": "fp32"},
        # a prefill batch of 4096 tokens with padding behind it, bf16 logits, the same rule
        {"name": "select_prefill", "op": "select", "tokens": 4096, "pad": 37, "experts": 384, "top_k": 8,
         "score": "sigmoid", "bias": True, "groups": 8, "limit": 4, "group_top": 2, "renormalize": True,
         "scale": 2.5, "dtype": "bf16"},
        # four batches of a training step: softmax over 896 experts, top-16, odd number of rows
        {"name": "select_training", "op": "select", "tokens": 16383, "pad": 0, "experts": 896, "top_k": 16,
         "score": "softmax", "bias": False, "groups": 1, "limit": 1, "group_top": 1, "renormalize": False,
         "scale": 1.0, "dtype": "fp32"},
        # the gradient of a small fine-tuning step: 300 tokens, 8 experts, top-2
        {"name": "select_backward_small", "op": "select_backward", "tokens": 293, "pad": 7, "experts": 8, "top_k": 2,
         "score": "sigmoid", "bias": True, "groups": 1, "limit": 1, "group_top": 1, "renormalize": True,
         "scale": 1.0, "dtype": "bf16"},
        # the gradient of the training step above: every logit of a row has one
        {"name": "select_backward_training", "op": "select_backward", "tokens": 16383, "pad": 0, "experts": 896,
         "top_k": 16, "score": "softmax", "bias": False, "groups": 1, "limit": 1, "group_top": 1,
         "renormalize": False, "scale": 1.0, "dtype": "fp32"},
        # a shared expert's gated w1||w3 for one decoded token
        {"name": "linear_one_token", "op": "linear", "m": 1, "n": 4096, "k": 7168, "gate": True, "dtype": "bf16"},
        # its w2 for an odd decode batch
        {"name": "linear_decode", "op": "linear", "m": 37, "n": 7168, "k": 2048, "gate": False, "dtype": "bf16"},
        # its gated w1||w3 over a large prefill batch
        {"name": "linear_prefill", "op": "linear", "m": 4096, "n": 4096, "k": 7168, "gate": True, "dtype": "bf16"},
        # a decode batch of 128 tokens, top-8, 224 of 384 experts resident
        {"name": "combine_decode", "op": "combine", "tokens": 128, "top_k": 8, "hidden": 7168, "resident": 224 / 384,
         "dtype": "bf16"},
        # a prefill batch with every expert resident, added up in fp32
        {"name": "combine_prefill", "op": "combine", "tokens": 4096, "top_k": 8, "hidden": 7168, "resident": 1.0,
         "dtype": "fp32"},
        # a small fine-tuning step: 301 tokens, top-2
        {"name": "combine_backward_small", "op": "combine_backward", "tokens": 301, "top_k": 2, "hidden": 1024,
         "resident": 1.0, "dtype": "bf16"},
        # a training step of 4096 tokens, top-8
        {"name": "combine_backward_training", "op": "combine_backward", "tokens": 4096, "top_k": 8, "hidden": 7168,
         "resident": 1.0, "dtype": "bf16"},
    ]


def _log(rng, low, high, step=1):
    """A multiple of `step` in [low, high], even over the logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("select", "select_backward", "linear", "combine", "combine_backward"))
    if op in ("select", "select_backward"):
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = groups * _log(rng, 4, 896 // groups)
        limit = rng.randint(1, groups)
        top_k = rng.randint(1, min(16, limit * experts // groups))
        return {"op": op, "tokens": _log(rng, 1, min(16384, MOST_LOGITS // experts - 8)), "pad": rng.choice((0, 0, 5)),
                "experts": experts, "top_k": top_k,
                "score": rng.choice(SCORES), "bias": rng.random() < 0.5, "groups": groups, "limit": limit,
                # a single renormalised weight is constant: its gradient is zero
                "group_top": rng.choice((1, 2)),
                "renormalize": rng.random() < 0.5 and (op == "select" or top_k > 1),
                "scale": rng.choice((1.0, 2.5)), "dtype": rng.choice(("fp32", "bf16"))}
    if op == "linear":
        gate = rng.random() < 0.5
        n, k = _log(rng, 16, 8192, 2 if gate else 1), _log(rng, 32, 8192, 32)
        return {"op": op, "m": _log(rng, 1, min(8192, MOST_LINEAR // (n * k))), "n": n, "k": k, "gate": gate,
                "dtype": rng.choice(("bf16", "bf16", "fp32"))}
    hidden, top_k = _log(rng, 64, 8192, 8), rng.choice((1, 2, 4, 6, 8, 16))
    return {"op": op, "tokens": _log(rng, 1, min(8192, MOST_ROUTED // (hidden * top_k))), "top_k": top_k,
            "hidden": hidden, "resident": rng.choice((1.0, 1.0, 224 / 384)), "dtype": rng.choice(("bf16", "fp32"))}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(shape, dtype=torch.float32, scale=1.0):
        t = torch.randn(shape, device=dev, dtype=torch.float32, generator=g)
        return (t.mul_(scale) if scale != 1.0 else t).to(dtype)

    op = case["op"]
    if op in ("select", "select_backward"):
        rows, experts = case["tokens"] + case["pad"], case["experts"]
        # experts differ in popularity; rows of padding are masked in full
        logits = normal((rows, experts), scale=1.5).add_(normal((1, experts), scale=0.5)).to(DTYPES[case["dtype"]])
        logits[case["tokens"]:] = float("-inf")
        state = dict(case, logits=logits, bias=normal((experts,), scale=0.05) if case["bias"] else None)
        if op == "select_backward":
            state["ids"] = _select(state)[0]
            state["dweights"] = normal((rows, case["top_k"]))
        return state
    if op == "linear":
        n, k = case["n"], case["k"]
        # weights of about k^-1/2, as trained ones are, so that the gate is neither shut nor open
        middle = 127 - round(math.log2(2.9 * math.sqrt(k)))
        return dict(case, x=normal((case["m"], k), torch.bfloat16),
                    codes=torch.randint(0, 256, (n, k // 2), device=dev, dtype=torch.uint8, generator=g),
                    scales=torch.randint(middle - 2, middle + 2, (n, k // GROUP), device=dev, dtype=torch.uint8,
                                         generator=g))
    tokens, top_k, hidden = case["tokens"], case["top_k"], case["hidden"]
    # routes sorted by expert, those of experts that are not resident left out
    ids = torch.randint(0, 384, (tokens * top_k,), device=dev, generator=g)
    resident = int(384 * case["resident"])
    order = torch.argsort(torch.where(ids < resident, ids, 384), stable=True)
    valid = int((ids < resident).sum())
    perm = torch.full((tokens * top_k,), -7, device=dev, dtype=torch.int32)
    perm[:valid] = order[:valid].int()
    rowpos = torch.full((tokens * top_k,), -1, device=dev, dtype=torch.int32)
    rowpos[order[:valid]] = torch.arange(valid, device=dev, dtype=torch.int32)
    state = dict(case, valid=valid, perm=perm, rowpos=rowpos.view(tokens, top_k),
                 y=normal((tokens * top_k, hidden), torch.bfloat16),
                 weights=torch.softmax(normal((tokens, top_k)), dim=1))
    if op == "combine_backward":
        state["dout"] = normal((tokens, hidden), DTYPES[case["dtype"]])
        # rows that no route has stay as they are
        state["dy"] = torch.zeros((tokens * top_k, hidden), device=dev, dtype=torch.bfloat16)
    return state


# ---- plain forms

def _finite(logits):
    """(fp32 logits, +inf taken as the largest number; which are masked: -inf and NaN)."""
    l = logits.float()
    masked = (l == float("-inf")) | torch.isnan(l)
    return l.clamp(max=FLOAT_MAX), masked


def _scores(l, masked, score):
    """Scores in l's type, 0 where masked."""
    if score == "sigmoid":
        return torch.where(masked, 0.0, torch.sigmoid(l))
    l = l.masked_fill(masked, float("-inf"))
    top = l.amax(dim=1, keepdim=True)
    terms = torch.exp(l - torch.where(top == float("-inf"), 0.0, top))
    return terms / terms.sum(dim=1, keepdim=True).clamp(min=1e-300 if l.dtype == torch.float64 else 1e-38)


def _select(state):
    l, masked = _finite(state["logits"])
    rows, experts = l.shape
    groups, per = state["groups"], experts // state["groups"]
    bias = state["bias"]
    scores = _scores(l.double(), masked, state["score"]) if bias is not None or groups > 1 else None
    value = l.double() if bias is None else scores + bias.double()
    value = value.masked_fill(masked, float("-inf"))
    if groups > state["limit"]:
        best = value if bias is not None or state["group_top"] == 1 else scores.masked_fill(masked, float("-inf"))
        best = best.view(rows, groups, per).sort(dim=2, descending=True).values[..., :state["group_top"]]
        shut = best[..., 0] == float("-inf")
        best = best.masked_fill(best == float("-inf"), 0.0).sum(dim=2).masked_fill(shut, float("-inf"))
        order = best.sort(dim=1, descending=True, stable=True).indices
        keep = torch.zeros((rows, groups), dtype=torch.bool, device=l.device)
        keep.scatter_(1, order[:, :state["limit"]], True)
        value = value.masked_fill(~keep.repeat_interleave(per, dim=1), float("-inf"))
    best, order = value.sort(dim=1, descending=True, stable=True)   # stable: equal values in order of their ids
    best, order = best[:, :state["top_k"]], order[:, :state["top_k"]]
    none = best == float("-inf")
    return order.masked_fill(none, -1).int(), _weights(state, l, masked, order, none)


def _weights(state, l, masked, order, none):
    w = _scores(l, masked, state["score"]).gather(1, order).masked_fill(none, 0.0)
    if state["renormalize"]:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-38)
    return w * state["scale"]


def _select_backward(state):
    l, masked = _finite(state["logits"])
    ids = state["ids"].long()
    none = ids < 0
    at = ids.clamp(min=0)
    s = _scores(l, masked, state["score"])
    picked = s.gather(1, at).masked_fill(none, 0.0)
    d = (state["dweights"] * state["scale"]).masked_fill(none, 0.0)
    if state["renormalize"]:
        total = picked.sum(dim=1, keepdim=True).clamp(min=1e-38)
        d = (d - (d * picked / total).sum(dim=1, keepdim=True)) / total
    ds = torch.zeros_like(l).scatter_add_(1, at, d.masked_fill(none, 0.0))
    if state["score"] == "sigmoid":
        dl = ds * s * (1.0 - s)
    elif state["renormalize"]:
        dl = ds * s   # the sum over a row of ds * s is zero
    else:
        dl = s * (ds - (ds * s).sum(dim=1, keepdim=True))
    return dl.to(state["logits"].dtype)


def _decode(codes, scales):
    nibbles = torch.stack((codes & 15, codes >> 4), dim=-1)
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device, dtype=torch.float32)
    values = grid[nibbles.long()].view(codes.shape[0], -1, GROUP)
    return (values * (scales.int() << 23).view(torch.float32).unsqueeze(-1)).view(codes.shape[0], -1)


def _plain(state):
    op = state["op"]
    if op == "select":
        return _select(state)
    if op == "select_backward":
        return _select_backward(state)
    if op == "linear":
        y = state["x"].float() @ _decode(state["codes"], state["scales"]).t()
        if state["gate"]:
            gate, up = y.chunk(2, dim=1)
            y = gate / (1.0 + torch.exp(-gate)) * up
        return y.to(DTYPES[state["dtype"]])
    rowpos, w = state["rowpos"], state["weights"]
    w = torch.where(rowpos < 0, 0.0, w)
    if op == "combine":
        rows = state["y"].float()[rowpos.clamp(min=0).long()]
        return (rows * w.unsqueeze(-1)).sum(dim=1).to(DTYPES[state["dtype"]])
    dout, valid = state["dout"].float(), state["valid"]
    dw = torch.stack([(dout * state["y"].float()[rowpos[:, s].clamp(min=0).long()]).sum(dim=1)
                      for s in range(state["top_k"])], dim=1)
    route = state["perm"][:valid].long()
    state["dy"][:valid] = (w.flatten()[route].unsqueeze(-1) * dout[route // state["top_k"]]).to(torch.bfloat16)
    return state["dy"], torch.where(rowpos < 0, 0.0, dw)


def run(state):
    if not own:
        return _plain(state)
    import mxfp4_routed_expert_topk_amd as moe
    op = state["op"]
    if op in ("select", "select_backward"):
        rule = dict(score=moe.MOE_SCORE_SIGMOID if state["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX,
                    renormalize=state["renormalize"], scale=state["scale"])
        if op == "select":
            return moe.router_select(state["logits"], state["top_k"], bias=state["bias"], num_groups=state["groups"],
                                     group_limit=state["limit"], group_top=state["group_top"], **rule)
        return moe.router_select_backward(state["dweights"], state["logits"], state["ids"], **rule)
    if op == "linear":
        return moe.mxfp4_linear(state["x"], state["codes"], state["scales"], gate=state["gate"],
                                dtype=DTYPES[state["dtype"]])
    if op == "combine":
        return moe.expert_combine(state["y"], state["rowpos"], state["weights"], dtype=DTYPES[state["dtype"]])
    return moe.expert_combine_backward(state["dout"], state["y"], state["rowpos"], state["perm"], state["weights"],
                                       dy=state["dy"])


# ---- what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("select", "select_backward"):
        rows = case["tokens"] + case["pad"]
        logits = rows * case["experts"] * (4 if case["dtype"] == "fp32" else 2)
        routes = rows * case["top_k"]
        if op == "select":
            # a score each, and a comparison of each with what is selected
            return {"bytes": logits + 8 * routes + 4 * case["experts"] * case["bias"],
                    "flops": 5 * rows * case["experts"]}
        # ids and weight gradients in, a gradient for every logit out; the
        # logits themselves count where every one of a row has a part
        dense = case["score"] == "softmax" and not case["renormalize"]
        picked = routes * (4 if case["dtype"] == "fp32" else 2)
        return {"bytes": logits + 8 * routes + (logits if dense else picked),
                "flops": (5 * rows * case["experts"] if dense else 8 * routes)}
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        out = m * (n // 2 if case["gate"] else n) * (4 if case["dtype"] == "fp32" else 2)
        return {"bytes": 2 * m * k + n * (k // 2 + k // GROUP) + out, "flops": 2 * m * n * k}
    tokens, routes, hidden = case["tokens"], case["tokens"] * case["top_k"], case["hidden"]
    valid = routes * int(384 * case["resident"]) / 384
    size = 4 if case["dtype"] == "fp32" else 2
    if op == "combine":
        return {"bytes": valid * hidden * 2 + tokens * hidden * size + 8 * routes, "flops": 2 * valid * hidden}
    # y, dout, the weights and rowpos in; dy and the weights' gradients out
    return {"bytes": 2 * valid * hidden * 2 + tokens * hidden * size + 12 * routes, "flops": 3 * valid * hidden}


# ---- the definitions in 64 bits

def _exact_select(case, logits, bias):
    """Row by row on the host: expert lists sorted by (value, id)."""
    l = np.minimum(logits.double().cpu().numpy(), float(FLOAT_MAX))
    open_ = ~(np.isnan(l) | np.isneginf(l))
    if case["score"] == "sigmoid":
        with np.errstate(over="ignore"):
            s = np.where(open_, 1.0 / (1.0 + np.exp(-np.where(open_, l, 0.0))), 0.0)
    else:
        top = np.where(open_, l, -np.inf).max(axis=1, initial=-FLOAT_MAX, keepdims=True)
        e = np.where(open_, np.exp(np.where(open_, l, top) - top), 0.0)
        s = e / np.maximum(e.sum(axis=1, keepdims=True), 1e-300)
    value = l if bias is None else s + bias.double().cpu().numpy()
    rows, experts = l.shape
    k, per = case["top_k"], experts // case["groups"]
    allowed = open_.copy()
    if case["groups"] > case["limit"]:
        grade = s if bias is None else value
        grade = np.sort(np.where(open_, grade, -np.inf).reshape(rows, -1, per), axis=2)[:, :, ::-1][:, :, :case["group_top"]]
        if bias is None and case["group_top"] == 1:
            total = np.where(open_, l, -np.inf).reshape(rows, -1, per).max(axis=2)
        else:
            total = np.where(np.isneginf(grade[:, :, 0]), -np.inf, np.where(np.isneginf(grade), 0.0, grade).sum(axis=2))
        rank = np.argsort(np.argsort(-total, axis=1, kind="stable"), axis=1)
        allowed &= np.repeat(rank < case["limit"], per, axis=1)
    value = np.where(allowed, value, -np.inf)
    ids = np.argsort(-value, axis=1, kind="stable")[:, :k]
    empty = ~np.take_along_axis(allowed, ids, axis=1)
    w = np.where(empty, 0.0, np.take_along_axis(s, ids, axis=1))
    if case["renormalize"]:
        w = w / np.maximum(w.sum(axis=1, keepdims=True), 1e-300)
    dev = logits.device
    return (torch.from_numpy(np.where(empty, -1, ids).astype(np.int32)).to(dev),
            torch.from_numpy(w * case["scale"]).to(dev))


def _exact_values(codes, scales):
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    c = np.empty((codes.shape[0], codes.shape[1] * 2), np.int64)
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    expo, man = (c >> 1) & 3, c & 1
    v = np.where(expo == 0, 0.5 * man, (2.0 + man) * np.exp2(expo - 2.0))
    v = np.where(c & 8, -v, v)
    return v * np.repeat(np.exp2(scales.astype(np.float64) - 127.0), GROUP, axis=1)


def exact(case, seed):
    state = prepare(case, seed)
    op = state["op"]
    if op == "select":
        return _exact_select(case, state["logits"], state["bias"])
    if op == "select_backward":
        # the weights as a function of the logits at these ids, differentiated by autograd
        l = state["logits"].double().nan_to_num(nan=-1e300, neginf=-1e300).requires_grad_()
        s = torch.special.expit(l) if case["score"] == "sigmoid" else torch.softmax(l, dim=1)
        live = (state["ids"] >= 0).double()
        w = torch.gather(s, 1, state["ids"].clamp(min=0).long()) * live
        if case["renormalize"]:
            w = w / (w.sum(dim=1, keepdim=True) + (live.sum(dim=1, keepdim=True) == 0))
        (w * case["scale"]).backward(state["dweights"].double())
        return l.grad
    if op == "linear":
        w = torch.from_numpy(_exact_values(state["codes"], state["scales"])).to(state["x"].device)
        y = torch.mm(state["x"].double(), w.t().contiguous())
        if case["gate"]:
            half = case["n"] // 2
            return y[:, :half] * torch.special.expit(y[:, :half]) * y[:, half:]
        return y
    rowpos, weights, y = state["rowpos"], state["weights"], state["y"]
    if op == "combine":
        out = torch.zeros((case["tokens"], case["hidden"]), device=y.device, dtype=torch.float64)
        for s in range(case["top_k"]):
            t = torch.nonzero(rowpos[:, s] >= 0).flatten()
            out[t] += weights[t, s].double().unsqueeze(1) * y[rowpos[t, s].long()].double()
        return out
    dy = torch.zeros(y.shape, device=y.device, dtype=torch.float64)
    dw = torch.zeros(weights.shape, device=y.device, dtype=torch.float64)
    for s in range(case["top_k"]):
        t = torch.nonzero(rowpos[:, s] >= 0).flatten()
        r = rowpos[t, s].long()
        d = state["dout"][t].double()
        dy[r] = weights[t, s].double().unsqueeze(1) * d
        dw[t, s] = (d * y[r].double()).sum(dim=1)
    return dy, dw
