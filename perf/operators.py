"""Measured cases of the MXFP4 quantiser and product and of the grouped products.

Operators, and the entry points that `run` calls where `own` is true:
  quantize    mxfp4_quantize, then mxfp4_dequantize (4-bit codes come back as the values they stand for)
  dequantize  mxfp4_dequantize
  matmul      mxfp4_matmul: both operands MXFP4, bf16 out
  grouped     grouped_matmul: rows sorted by expert times that expert's bf16 matrix
  backward    grouped_matmul_backward: gradients of the rows and of every expert's matrix

Where `own` is false the same results are computed from elementary torch
operations in fp32, rounded once at the end.
"""
import math

import numpy as np
import torch

own = False

GROUP = 32                                             # elements per E8M0 scale
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)        # magnitudes of the E2M1 codes 0..7
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}

# Sizes of the layer's own workloads: hidden 7168, intermediate 2048 (a fused
# w1||w3 matrix is [4096, 7168], w2 [7168, 2048]), 224 resident of 384 experts.
MOST_ELEMENTS = 16384 * 7168
MOST_MATMUL = 4096 * 4096 * 7168
MOST_GROUPED = 32768 * 4096 * 7168
MOST_BACKWARD = 12288 * 4096 * 7168
MOST_WEIGHTS = 224 * 7168 * 2048
MOST_WEIGHTS_BACKWARD = 32 * 4096 * 7168


def listed():
    return [
        # a decode batch's activations before an MXFP4 product
        {"name": "quantize_decode", "op": "quantize", "rows": 16, "cols": 7168, "dtype": "bf16"},
        # four experts' fp32 master w1||w3 on their way to the layer's plan
        {"name": "quantize_weights", "op": "quantize", "rows": 16384, "cols": 7168, "dtype": "fp32"},
        # one small matrix read back for inspection
        {"name": "dequantize_small", "op": "dequantize", "rows": 384, "cols": 2048, "dtype": "fp32"},
        # two experts' w2 read back as bf16
        {"name": "dequantize_weights", "op": "dequantize", "rows": 14336, "cols": 2048, "dtype": "bf16"},
        # a shared expert's w1||w3 for one decoded token
        {"name": "matmul_one_token", "op": "matmul", "m": 1, "n": 4096, "k": 7168},
        # its w2 for an odd decode batch
        {"name": "matmul_decode", "op": "matmul", "m": 37, "n": 7168, "k": 2048},
        # its w1||w3 over a large prefill batch
        {"name": "matmul_prefill", "op": "matmul", "m": 4096, "n": 4096, "k": 7168},
        # the smallest layer: 16 tokens, 8 experts, top-2
        {"name": "grouped_tiny", "op": "grouped", "rows": 32, "pad": 0, "experts": 8, "n": 256, "k": 256, "skew": 0.0},
        # bf16 w2 of a decode batch: 128 tokens, top-8, the routes that are resident
        {"name": "grouped_decode", "op": "grouped", "rows": 597, "pad": 427, "experts": 224, "n": 7168, "k": 2048,
         "skew": 0.0},
        # bf16 w1||w3 of 4096 tokens, top-8, Zipf popularity
        {"name": "grouped_prefill", "op": "grouped", "rows": 32768, "pad": 0, "experts": 64, "n": 4096, "k": 7168,
         "skew": 1.2},
        # a small fine-tuning step: 300 tokens, top-2, bf16 gradients
        {"name": "backward_small", "op": "backward", "rows": 593, "pad": 7, "experts": 8, "n": 768, "k": 1024,
         "skew": 1.2, "dw": "bf16"},
        # a training step of 1536 tokens, top-8, fp32 weight gradients
        {"name": "backward_large", "op": "backward", "rows": 12288, "pad": 0, "experts": 32, "n": 4096, "k": 7168,
         "skew": 0.0, "dw": "fp32"},
    ]


def _log(rng, low, high, step=1):
    """A multiple of `step` in [low, high], even over the logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("quantize", "dequantize", "matmul", "grouped", "backward"))
    if op in ("quantize", "dequantize"):
        cols = _log(rng, 32, 16384, 32)
        return {"op": op, "rows": _log(rng, 1, min(65536, MOST_ELEMENTS // cols)), "cols": cols,
                "dtype": rng.choice(("bf16", "fp32"))}
    if op == "matmul":
        n, k = _log(rng, 16, 8192), _log(rng, 32, 8192, 32)
        return {"op": op, "m": _log(rng, 1, min(8192, MOST_MATMUL // (n * k))), "n": n, "k": k}
    n, k = _log(rng, 64, 7168, 8), _log(rng, 64, 7168, 8)
    most = MOST_GROUPED if op == "grouped" else MOST_BACKWARD
    weights = MOST_WEIGHTS if op == "grouped" else MOST_WEIGHTS_BACKWARD
    experts = _log(rng, 1, min(224, weights // (n * k)))
    case = {"op": op, "rows": _log(rng, 1, min(32768, most // (n * k))), "pad": rng.choice((0, 0, rng.randint(1, 300))),
            "experts": experts, "n": n, "k": k, "skew": rng.choice((0.0, 0.0, 0.6, 1.2))}
    if op == "backward":
        case["dw"] = rng.choice(("fp32", "bf16"))
    return case


def _popularity(case):
    p = np.arange(1, case["experts"] + 1, dtype=np.float64) ** -case["skew"]
    return p / p.sum()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(shape, dtype, scale=1.0):
        t = torch.randn(shape, device=dev, dtype=dtype, generator=g)
        return t.mul_(scale) if scale != 1.0 else t

    def mxfp4(rows, cols):
        codes = torch.randint(0, 256, (rows, cols // 2), device=dev, dtype=torch.uint8, generator=g)
        scales = torch.randint(118, 133, (rows, cols // GROUP), device=dev, dtype=torch.uint8, generator=g)
        return codes, scales

    op = case["op"]
    if op == "quantize":
        # rows of different magnitude, a few large elements, some groups of zeros
        x = normal((case["rows"], case["cols"]), DTYPES[case["dtype"]])
        size = torch.exp2(torch.randint(-6, 4, (case["rows"], 1), device=dev, generator=g).float())
        x.mul_(size.to(x.dtype))
        groups = x.view(case["rows"], -1, GROUP)
        pick = torch.rand(groups.shape[:2], device=dev, generator=g)
        groups[..., 5].mul_(torch.where(pick > 0.9, 20.0, 1.0).to(x.dtype))
        groups.mul_((pick > 0.01).to(x.dtype).unsqueeze(-1))
        return {"op": op, "x": x}
    if op == "dequantize":
        codes, scales = mxfp4(case["rows"], case["cols"])
        return {"op": op, "codes": codes, "scales": scales, "dtype": DTYPES[case["dtype"]]}
    if op == "matmul":
        return {"op": op, "a": mxfp4(case["m"], case["k"]), "b": mxfp4(case["n"], case["k"])}
    rows, total, n, k = case["rows"], case["rows"] + case["pad"], case["n"], case["k"]
    counts = np.random.default_rng(seed).multinomial(rows, _popularity(case))
    np.random.default_rng(seed + 1).shuffle(counts)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    state = {"op": op, "counts": [int(c) for c in counts], "rows": rows,
             "offsets": torch.from_numpy(offsets).to(dev),
             "x": normal((total, k), torch.bfloat16),
             "w": normal((case["experts"], n, k), torch.bfloat16, k ** -0.5)}
    # rows behind the last group belong to nobody and stay as they are
    if op == "grouped":
        state["out"] = torch.zeros((total, n), device=dev, dtype=torch.bfloat16)
    else:
        state["dy"] = normal((total, n), torch.bfloat16)
        state["dx"] = torch.zeros((total, k), device=dev, dtype=torch.bfloat16)
        state["dw"] = DTYPES[case["dw"]]
    return state


# ---- plain forms

def _grid(like):
    return torch.tensor(GRID + tuple(-v for v in GRID), device=like.device, dtype=torch.float32)


def _power(e):
    return ((e + 127) << 23).view(torch.float32)      # 2^e, the exponent bits of a float


def _decode(codes, scales):
    nibbles = torch.stack((codes & 15, codes >> 4), dim=-1)
    values = _grid(codes)[nibbles.long()].view(codes.shape[0], -1, GROUP)
    return (values * _power(scales.int() - 127).unsqueeze(-1)).view(codes.shape[0], -1)


def _quantize(x):
    groups = x.float().view(x.shape[0], -1, GROUP)
    amax = groups.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, -125).clamp(-125, 125)
    v = groups * _power(-e).unsqueeze(-1)
    a = v.abs()
    # nearest grid point; a tie goes to the code with an even last bit
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int() + 8 * (v < 0).int()).view(x.shape)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8), (e + 127).to(torch.uint8)


def _plain(state):
    op = state["op"]
    if op == "quantize":
        return _decode(*_quantize(state["x"])).to(torch.bfloat16)
    if op == "dequantize":
        return _decode(state["codes"], state["scales"]).to(state["dtype"])
    if op == "matmul":
        return (_decode(*state["a"]) @ _decode(*state["b"]).t()).to(torch.bfloat16)
    rows, counts, w = state["rows"], state["counts"], state["w"]
    xs = state["x"][:rows].split(counts)
    if op == "grouped":
        state["out"][:rows] = torch.cat([x.float() @ m.float().t() for x, m in zip(xs, w)]).to(torch.bfloat16)
        return state["out"]
    dys = state["dy"][:rows].split(counts)
    state["dx"][:rows] = torch.cat([dy.float() @ m.float() for dy, m in zip(dys, w)]).to(torch.bfloat16)
    return state["dx"], torch.stack([(dy.float().t() @ x.float()).to(state["dw"]) for dy, x in zip(dys, xs)])


def run(state):
    if not own:
        return _plain(state)
    import mxfp4_routed_expert_topk_amd as moe
    op = state["op"]
    if op == "quantize":
        return moe.mxfp4_dequantize(*moe.mxfp4_quantize(state["x"]))
    if op == "dequantize":
        return moe.mxfp4_dequantize(state["codes"], state["scales"], dtype=state["dtype"])
    if op == "matmul":
        return moe.mxfp4_matmul(*state["a"], *state["b"])
    if op == "grouped":
        return moe.grouped_matmul(state["x"], state["w"], state["offsets"], out=state["out"])
    return moe.grouped_matmul_backward(state["dy"], state["x"], state["w"], state["offsets"], dx=state["dx"],
                                       dw_dtype=state["dw"])


# ---- what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("quantize", "dequantize"):
        n = case["rows"] * case["cols"]
        size = 4 if case["dtype"] == "fp32" else 2
        packed = n // 2 + n // GROUP
        # quantize: x in, codes and scales out, and the bf16 values they stand for
        return {"bytes": n * size + packed + (2 * n if op == "quantize" else 0), "flops": 2 * n}
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * (k // 2 + k // GROUP) + 2 * m * n, "flops": 2 * m * n * k}
    rows, n, k = case["rows"], case["n"], case["k"]
    # experts that get a row, on average over the routing
    touched = float((1.0 - (1.0 - _popularity(case)) ** rows).sum())
    weights, acts = 2 * touched * n * k, 2 * rows * (n + k)
    if op == "grouped":
        return {"bytes": weights + acts, "flops": 2.0 * rows * n * k}
    grads = (4 if case["dw"] == "fp32" else 2) * case["experts"] * n * k
    return {"bytes": weights + acts + 2 * rows * k + grads, "flops": 4.0 * rows * n * k}


# ---- the definitions in 64 bits

def _exact_values(codes, scales):
    sign = 1.0 - 2.0 * ((codes.unsqueeze(-1) >> torch.tensor([3, 7], device=codes.device)) & 1).double()
    expo = (codes.unsqueeze(-1) >> torch.tensor([1, 5], device=codes.device)) & 3
    man = ((codes.unsqueeze(-1) >> torch.tensor([0, 4], device=codes.device)) & 1).double()
    size = torch.where(expo == 0, 0.5 * man, (1.0 + 0.5 * man) * torch.exp2(expo.double() - 1.0))
    scale = torch.exp2(scales.double() - 127.0).repeat_interleave(GROUP, dim=1)
    return (sign * size).flatten(1) * scale


def _exact_rounded(x):
    groups = x.double().view(-1, GROUP)
    amax = groups.abs().amax(1, keepdim=True)
    e = torch.floor(torch.log2(amax)).clamp(-123, 127) - 2
    e = torch.where(torch.exp2(e + 3) <= amax, e + 1, e)      # a logarithm just below a whole number
    e = torch.where(torch.exp2(e + 2) > amax, e - 1, e).clamp(-125, 125)
    v = groups / torch.exp2(e)
    # spacing of the grid: 1/2 below 2, 1 below 4, 2 above
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0))
    return ((torch.round(v / step) * step).clamp(-6, 6) * torch.exp2(e)).view(x.shape)


def exact(case, seed):
    state = prepare(case, seed)
    op = state["op"]
    if op == "quantize":
        return _exact_rounded(state["x"])
    if op == "dequantize":
        return _exact_values(state["codes"], state["scales"])
    if op == "matmul":
        a, b = _exact_values(*state["a"]), _exact_values(*state["b"])
        return torch.mm(a, b.t().contiguous())
    bounds = state["offsets"].tolist()
    x, w = state["x"], state["w"]
    if op == "grouped":
        y = torch.zeros(state["out"].shape, device=x.device, dtype=torch.float64)
        for i in range(case["experts"]):
            r = slice(bounds[i], bounds[i + 1])
            y[r] = torch.mm(x[r].double(), w[i].double().t().contiguous())
        return y
    dy = state["dy"]
    dx = torch.zeros(state["dx"].shape, device=x.device, dtype=torch.float64)
    dw = torch.empty(w.shape, device=x.device, dtype=torch.float64)
    for i in range(case["experts"]):
        r = slice(bounds[i], bounds[i + 1])
        dx[r] = torch.mm(dy[r].double(), w[i].double())
        dw[i] = torch.mm(dy[r].double().t().contiguous(), x[r].double())
    return dx, dw
