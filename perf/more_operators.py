"""What is measured of the feed-forward operators: the cases, their inputs,
each operator in its plain form (elementary torch operations in 32 bits,
rounded once at the end), the framework's calls, and the definitions in 64
bits.

Four operators, which are a feed-forward block forward and backward in bf16
or fp16, each a product with what stands next to it done in the same pass:

  linear           C = act(A B + A2 B2 + bias) + residual; the second product,
                   the bias, the activation and the residual may be absent,
                   and Z, what the activation is taken of, may be kept.  B is
                   N x K (layout "RC", as a layer's weight lies) or K x N ("RR",
                   the same weight in the gradient of the layer's input).
  gated            H = act(X Wg^T + bg) * (X Wu^T + bu); G and U, the two
                   factors' arguments, may be kept.
  gated_backward   with dH = dY W: dG = dH * U * act'(G), dU = dH * act(G), and
                   H = act(G) * U again; without U: dG = dH * act'(G).
  weight_gradient  dW = dC^T A in fp32, and db, the sums of dC's columns.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
ACTIVATIONS = ("relu", "gelu", "gelu_tanh", "silu")
# Most multiply-adds of a drawn case (under the largest listed one).
MOST_MACS = 8192 * 8192 * 8192


def listed():
    return [
        # one token through a layer with an activation: launch and weight latency
        {"name": "linear_token", "op": "linear", "M": 1, "N": 4096, "K": 4096, "x": "bf16", "layout": "RC", "bias": True,
         "act": "gelu", "residual": False, "pair": False, "keep": False},
        # a decoding batch of 64 sequences through the block's last layer: the weights' bytes
        {"name": "linear_batch", "op": "linear", "M": 64, "N": 8192, "K": 8192, "x": "bf16", "layout": "RC", "bias": False,
         "act": "none", "residual": True, "pair": False, "keep": False},
        # a mixed batch of odd length, rows that start on no common boundary, ragged in every direction
        {"name": "linear_odd", "op": "linear", "M": 500, "N": 4104, "K": 4100, "x": "f16", "layout": "RC", "bias": True,
         "act": "gelu_tanh", "residual": True, "pair": False, "keep": False},
        # a training batch through a layer whose gradient will want Z: matrix cores
        {"name": "linear_train", "op": "linear", "M": 8192, "N": 8192, "K": 8200, "x": "bf16", "layout": "RC", "bias": True,
         "act": "gelu_tanh", "residual": False, "pair": False, "keep": True},
        # the gradient of a gated block's input, from both of its halves, added to the residual's
        {"name": "linear_two_products", "op": "linear", "M": 8192, "N": 4096, "K": 8192, "x": "bf16", "layout": "RR",
         "bias": False, "act": "none", "residual": True, "pair": True, "keep": False},
        # one token of a decoding step through a gated block: the weights' bytes
        {"name": "gated_token", "op": "gated", "M": 1, "N": 8192, "K": 4096, "x": "bf16", "act": "silu", "bias": False,
         "keep": False},
        # a short prompt
        {"name": "gated_prompt", "op": "gated", "M": 500, "N": 8192, "K": 4096, "x": "bf16", "act": "silu", "bias": False,
         "keep": False},
        # a training batch, with what the backward pass wants
        {"name": "gated_train", "op": "gated", "M": 8192, "N": 8192, "K": 4096, "x": "bf16", "act": "silu", "bias": False,
         "keep": True},
        # the backward pass of a short, odd batch through a layer with an activation
        {"name": "gated_backward_short", "op": "gated_backward", "M": 65, "N": 4104, "K": 1024, "x": "f16", "act": "gelu",
         "gate": False, "keep": False},
        # the backward pass of a training batch, with H again for the next weight's gradient
        {"name": "gated_backward_step", "op": "gated_backward", "M": 8192, "N": 8192, "K": 4096, "x": "bf16", "act": "silu",
         "gate": True, "keep": True},
        # a weight's gradient from a short, odd batch: the bytes of the result
        {"name": "weight_gradient_short", "op": "weight_gradient", "M": 65, "N": 4104, "K": 4096, "x": "bf16", "bias": True},
        # a weight's gradient from a training batch: matrix cores
        {"name": "weight_gradient_step", "op": "weight_gradient", "M": 8192, "N": 8192, "K": 4096, "x": "bf16",
         "bias": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _tokens(rng):
    """1 to 8192, spread over the logarithm, half of them multiples of 16."""
    n = _log(rng, 1, 8192)
    return max(16, n // 16 * 16) if rng.random() < 0.5 else n


def _width(rng):
    """A layer's width, 64 to 8192, spread over the logarithm: multiples of 128 or of 8, as layers have them, but one in eight any."""
    n, kind = _log(rng, 64, 8192), rng.random()
    return n if kind < 0.125 else max(64, n // 8 * 8) if kind < 0.5 else max(128, n // 128 * 128)


def draw(rng):
    op = rng.choice(("linear", "linear", "gated", "gated_backward", "weight_gradient"))
    M, N, K = _tokens(rng), _width(rng), _width(rng)
    case = {"op": op, "M": M, "N": N, "K": K, "x": rng.choice(("bf16", "bf16", "f16"))}
    if op == "linear":
        case["layout"] = rng.choice(("RC", "RC", "RR"))
        case["act"] = "none" if case["layout"] == "RR" else rng.choice(("none",) + ACTIVATIONS)
        case["bias"] = case["layout"] == "RC" and rng.random() < 0.5
        case["residual"] = rng.random() < 0.5
        case["pair"] = case["layout"] == "RR" and rng.random() < 0.5
        case["keep"] = case["act"] != "none" and rng.random() < 0.5
    elif op == "weight_gradient":
        case["bias"] = rng.random() < 0.5
    else:
        case["act"] = rng.choice(ACTIVATIONS + ("silu", "silu"))
        case["keep"] = rng.random() < 0.5
        if op == "gated":
            case["bias"] = rng.random() < 0.3
        else:
            case["gate"] = rng.random() < 0.7
    products = 2 if op == "gated" or case.get("pair") else 1
    case["N"] = min(N, max(64, MOST_MACS // (products * M * K)))
    return case


# ---- inputs -----------------------------------------------------------------

def _values(g, rows, cols, dtype, size=1.0):
    """Activations: normal, with columns of unlike sizes and a few large ones."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    s = torch.exp(0.3 * torch.randn((cols,), generator=g, device="cuda"))
    s = torch.where(torch.rand((cols,), generator=g, device="cuda") < 0.002, s * 5, s)
    return (x * s * size).to(dtype)


def _weight(g, rows, cols, inputs, dtype):
    """A layer's weight: each output is about 1 on inputs of about 1."""
    return (torch.randn((rows, cols), generator=g, device="cuda") / math.sqrt(inputs)).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, t = dict(case), TYPES[case["x"]]
    M, N, K = c["M"], c["N"], c["K"]
    s = {"case": c}
    if c["op"] == "linear":
        shape = (N, K) if c["layout"] == "RC" else (K, N)
        s["a"], s["b"] = _values(g, M, K, t), _weight(g, *shape, K, t)
        s["pair"] = (_values(g, M, K, t), _weight(g, *shape, K, t)) if c["pair"] else None
        s["bias"] = 0.2 * torch.randn((N,), generator=g, device="cuda") if c["bias"] else None
        s["residual"] = _values(g, M, N, t, 2.0) if c["residual"] else None
    elif c["op"] == "gated":
        s["x"], s["wg"], s["wu"] = _values(g, M, K, t), _weight(g, N, K, K, t), _weight(g, N, K, K, t)
        s["bg"] = (0.2 * torch.randn((N,), generator=g, device="cuda")).to(t) if c["bias"] else None
        s["bu"] = (0.2 * torch.randn((N,), generator=g, device="cuda")).to(t) if c["bias"] else None
    elif c["op"] == "gated_backward":
        s["dy"], s["w"] = _values(g, M, K, t, 0.01), _weight(g, K, N, N, t)
        s["g"], s["u"] = _values(g, M, N, t), _values(g, M, N, t) if c["gate"] else None
    else:
        s["dc"], s["a"] = _values(g, M, N, t, 0.01), _values(g, M, K, t)
    return s


# ---- the plain forms --------------------------------------------------------

_ROOT = math.sqrt(2.0 / math.pi)


def _act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return torch.clamp_min(z, 0.0)
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1.0 + torch.tanh(_ROOT * (z + 0.044715 * z * z * z)))


def _slope(z, name):
    """The activation's derivative (relu's is 0 at 0)."""
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    t = torch.tanh(_ROOT * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _ROOT * (1.0 + 3 * 0.044715 * z * z)


def _linear(s):
    c, t = s["case"], s["a"].dtype
    turn = (lambda b: b.t()) if c["layout"] == "RC" else (lambda b: b)
    z = s["a"].float() @ turn(s["b"].float())
    if s["pair"] is not None:
        z = z + s["pair"][0].float() @ turn(s["pair"][1].float())
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return (y.to(t), z.to(t)) if c["keep"] else y.to(t)


def _gated(s):
    c, t, x = s["case"], s["x"].dtype, s["x"].float()
    g, u = x @ s["wg"].float().t(), x @ s["wu"].float().t()
    if s["bg"] is not None:
        g, u = g + s["bg"].float(), u + s["bu"].float()
    h = (_act(g, c["act"]) * u).to(t)
    return (h, g.to(t), u.to(t)) if c["keep"] else h


def _gated_backward(s):
    c, t = s["case"], s["dy"].dtype
    dh, g = s["dy"].float() @ s["w"].float(), s["g"].float()
    if s["u"] is None:
        out = ((dh * _slope(g, c["act"])).to(t),)
        return out + (_act(g, c["act"]).to(t),) if c["keep"] else out[0]
    u, a = s["u"].float(), _act(g, c["act"])
    out = ((dh * u * _slope(g, c["act"])).to(t), (dh * a).to(t))
    return out + ((a * u).to(t),) if c["keep"] else out


def _weight_gradient(s):
    dc = s["dc"].float()
    dw = dc.t() @ s["a"].float()
    return (dw, s["dc"].double().sum(0).float()) if s["case"]["bias"] else dw


def _own(s):
    from software_pipelined_tiled_02_amd import binding
    c = s["case"]
    if c["op"] == "linear":
        return binding.linear(s["a"], s["b"], layout=c["layout"], bias=s["bias"], activation=c["act"], residual=s["residual"],
                              pair=s["pair"], keep=c["keep"])
    if c["op"] == "gated":
        return binding.gated(s["x"], s["wg"], s["wu"], gate_bias=s["bg"], up_bias=s["bu"], activation=c["act"], keep=c["keep"])
    if c["op"] == "gated_backward":
        return binding.gated_backward(s["dy"], s["w"], s["g"], s["u"], activation=c["act"], keep=c["keep"])
    return binding.weight_gradient(s["dc"], s["a"], bias=c["bias"])


def run(state):
    if own:
        return _own(state)
    return {"linear": _linear, "gated": _gated, "gated_backward": _gated_backward,
            "weight_gradient": _weight_gradient}[state["case"]["op"]](state)


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    c = case
    M, N, K = c["M"], c["N"], c["K"]
    if c["op"] == "linear":
        products = 2 if c["pair"] else 1
        values = products * (M * K + N * K) + M * N * (1 + int(c["residual"]) + int(c["keep"]))
        return {"bytes": 2 * values + (4 * N if c["bias"] else 0), "flops": 2 * products * M * N * K}
    if c["op"] == "gated":
        values = M * K + 2 * N * K + M * N * (3 if c["keep"] else 1) + (2 * N if c["bias"] else 0)
        return {"bytes": 2 * values, "flops": 4 * M * N * K}
    if c["op"] == "gated_backward":
        values = M * K + N * K + M * N * ((4 if c["gate"] else 2) + int(c["keep"]))
        return {"bytes": 2 * values, "flops": 2 * M * N * K}
    return {"bytes": 2 * M * (N + K) + 4 * N * K + (4 * N if c["bias"] else 0), "flops": 2 * M * N * K}


# ---- the definitions in 64 bits ---------------------------------------------

def _exact_act(z, name):
    """(act(z), act'(z))"""
    one = torch.ones_like(z)
    if name == "none":
        return z, one
    if name == "relu":
        on = torch.where(z > 0, one, torch.zeros_like(z))
        return torch.where(z > 0, z, torch.zeros_like(z)), on
    if name == "gelu":
        half = 0.5 * torch.special.erfc(-z / 2.0 ** 0.5)              # the normal distribution's function
        return z * half, half + z * torch.exp(-z * z / 2) / (2 * math.pi) ** 0.5
    q, dq = (z, one) if name == "silu" else (2 * _ROOT * (z + 0.044715 * z ** 3), 2 * _ROOT * (1 + 0.134145 * z ** 2))
    s = torch.sigmoid(q)                                             # (1 + tanh(q / 2)) / 2
    return z * s, s + z * s * (1 - s) * dq


def exact(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in prepare(case, seed).items()}
    c = s["case"]
    if c["op"] == "linear":
        pairs = [(s["a"], s["b"])] + ([(s["pair"][0].double(), s["pair"][1].double())] if s["pair"] is not None else [])
        z = torch.zeros((c["M"], c["N"]), dtype=torch.float64, device="cuda") if s["bias"] is None else s["bias"].expand(c["M"], -1)
        for a, b in pairs:
            z = torch.addmm(z, a, b.t().contiguous() if c["layout"] == "RC" else b)
        y = _exact_act(z, c["act"])[0]
        y = y if s["residual"] is None else s["residual"] + y
        return (y, z) if c["keep"] else y
    if c["op"] == "gated":
        both = torch.mm(s["x"], torch.cat((s["wg"], s["wu"])).t().contiguous())
        g, u = both[:, :c["N"]], both[:, c["N"]:]
        if s["bg"] is not None:
            g, u = g + s["bg"], u + s["bu"]
        h = u * _exact_act(g, c["act"])[0]
        return (h, g, u) if c["keep"] else h
    if c["op"] == "gated_backward":
        dh, (a, d) = torch.mm(s["dy"], s["w"]), _exact_act(s["g"], c["act"])
        if s["u"] is None:
            return (dh * d, a) if c["keep"] else dh * d
        out = (dh * d * s["u"], dh * a)
        return out + (s["u"] * a,) if c["keep"] else out
    dw = torch.mm(s["dc"].t().contiguous(), s["a"])
    if not c["bias"]:
        return dw
    return dw, torch.mv(s["dc"].t().contiguous(), torch.ones((c["M"],), dtype=torch.float64, device="cuda"))
