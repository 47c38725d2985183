"""What is measured of the 8-bit floating-point operators: the cases, their
inputs, each operator in its plain form (elementary torch operations in 32
bits, rounded once at the end), the framework's calls, and the definitions in
64 bits.

Four operators, which are the way of one linear layer through 8 bits:

  product      C[i][j] = sum over blocks kb of SA[i][kb] SB[j][kb] *
               sum over k in block kb of A[i][k] B[j][k]; A (M x K) and B
               (N x K) hold 8-bit floats, a block is 128 values of k, and SB
               has one row for each 128 rows of B ("tile") or each ("row").
  quantize     per block of 128 values ("row") or of 128 x 128 ("tile"):
               s = max(amax |x| / top, 2^-126), q = fp8(x * (1 / s)); `top` is the
               type's largest value, and `pow2` rounds s up to a power of two.
               `transpose` also gives x transposed, quantised along its rows.
  rms          h = x + residual, rounded to x's type; y = h * rstd * w with
               rstd = 1 / sqrt(mean(h^2) + eps); y quantised by rows.
  rms_backward dx = dh + rstd (w dy - h rstd^2 mean(w dy h)),
               dw = sum over rows of dy h rstd.

Rows of 8-bit matrices start on 16 bytes, as the quantisers lay them out.
"""
import math

import torch

own = False

BLOCK = 128
EPS = 1e-6
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# Most multiply-adds of a drawn product (under the largest listed one) and
# most elements of a drawn quantisation or norm.
MOST_MACS = 8192 * 8192 * 8192
MOST_ELEMENTS = 8192 * 8192


def listed():
    return [
        # one token through one projection: launch and weight latency
        {"name": "product_token", "op": "product", "M": 1, "N": 4096, "K": 4096, "a": "e4m3", "b": "e4m3",
         "sb": "tile", "out": "bf16"},
        # a decoding batch of 64 sequences: the weights' bytes
        {"name": "product_skinny", "op": "product", "M": 64, "N": 8192, "K": 8192, "a": "e4m3", "b": "e4m3",
         "sb": "tile", "out": "bf16"},
        # a mixed batch of odd length, ragged in every direction
        {"name": "product_odd", "op": "product", "M": 500, "N": 4104, "K": 4100, "a": "e4m3", "b": "e4m3",
         "sb": "tile", "out": "f16"},
        # a long prompt or a training batch: matrix cores
        {"name": "product_prompt", "op": "product", "M": 8192, "N": 8192, "K": 8200, "a": "e4m3", "b": "e4m3",
         "sb": "tile", "out": "bf16"},
        # a weight's gradient: both operands scaled along the tokens, fp32 out
        {"name": "product_weight_gradient", "op": "product", "M": 4096, "N": 4096, "K": 8200, "a": "e5m2", "b": "e4m3",
         "sb": "row", "out": "f32"},
        # a decoding batch's activations: launch latency
        {"name": "quantize_batch", "op": "quantize", "M": 16, "K": 4096, "x": "bf16", "fp8": "e4m3", "block": "row",
         "pow2": False, "transpose": False},
        # a training step's output gradient, for both products of the backward pass
        {"name": "quantize_both_ways", "op": "quantize", "M": 8192, "K": 8192, "x": "bf16", "fp8": "e5m2",
         "block": "row", "pow2": False, "transpose": True},
        # a weight after its update, for the forward and the backward product
        {"name": "quantize_weight", "op": "quantize", "M": 4104, "K": 8200, "x": "f32", "fp8": "e4m3", "block": "tile",
         "pow2": False, "transpose": True},
        # one token of a decoding step: latency
        {"name": "rms_token", "op": "rms", "M": 1, "D": 8192, "x": "bf16", "w": "bf16", "residual": True},
        # a prompt or a training batch
        {"name": "rms_prompt", "op": "rms", "M": 8192, "D": 8192, "x": "bf16", "w": "bf16", "residual": True},
        # the backward pass of a short, odd batch
        {"name": "rms_backward_short", "op": "rms_backward", "M": 65, "D": 4104, "x": "bf16", "w": "f32", "dh": False},
        # the backward pass of a training batch
        {"name": "rms_backward_step", "op": "rms_backward", "M": 8192, "D": 4096, "x": "bf16", "w": "bf16", "dh": True},
    ]


def _spread(rng, lo, hi, multiple):
    """A size between lo and hi, spread over its logarithm: half of them multiples of `multiple`."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        n = max(multiple, n // multiple * multiple)
    return min(max(n, lo), hi)


def draw(rng):
    op = rng.choice(("product", "product", "quantize", "rms", "rms_backward"))
    if op == "product":
        gradient = rng.random() < 0.3
        M, N, K = _spread(rng, 1, 8192, 16), _spread(rng, 64, 8192, 128), _spread(rng, 64, 8200, 128)
        N = min(N, max(64, MOST_MACS // (M * K)))
        return {"op": op, "M": M, "N": N, "K": K, "a": rng.choice(("e4m3", "e5m2")) if gradient else "e4m3", "b": "e4m3",
                "sb": "row" if gradient else "tile",
                "out": "f32" if gradient else rng.choice(("bf16", "bf16", "f16", "f32"))}
    M, D = _spread(rng, 1, 8192, 16), _spread(rng, 64, 16384, 128)
    D = min(D, max(64, MOST_ELEMENTS // M))
    x = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "quantize":
        return {"op": op, "M": M, "K": D, "x": x, "fp8": rng.choice(("e4m3", "e5m2")), "block": rng.choice(("row", "tile")),
                "pow2": rng.random() < 0.3, "transpose": rng.random() < 0.5}
    w = rng.choice((x, "f32"))
    if op == "rms":
        return {"op": op, "M": M, "D": D, "x": x, "w": w, "residual": rng.random() < 0.7}
    return {"op": op, "M": M, "D": D, "x": x, "w": w, "dh": rng.random() < 0.5}


def _blocks(n):
    return -(-n // BLOCK)


# ---- inputs -----------------------------------------------------------------

def _values(g, rows, cols, spread=0.5):
    """Activations, weights or gradients: normal, with columns of unlike sizes and a few large ones."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    size = torch.exp(spread * torch.randn((cols,), generator=g, device="cuda"))
    size = torch.where(torch.rand((cols,), generator=g, device="cuda") < 0.002, size * 20, size)
    return x * size


def _rows16(q):
    """q with rows that start on 16 bytes."""
    pad = torch.zeros((q.shape[0], -(-q.shape[1] // 16) * 16), dtype=torch.uint8, device=q.device)
    pad[:, : q.shape[1]] = q.view(torch.uint8)
    return pad.view(q.dtype)[:, : q.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    if c["op"] == "product":
        tile = c["sb"] == "tile"
        qa, sa = _quantize(_values(g, c["M"], c["K"]), c["a"], 1, False)
        qb, sb = _quantize(_values(g, c["N"], c["K"], 0.2) * 0.02, c["b"], BLOCK if tile else 1, False)
        return {"case": c, "a": _rows16(qa), "sa": sa, "b": _rows16(qb), "sb": sb}
    if c["op"] == "quantize":
        return {"case": c, "x": _values(g, c["M"], c["K"]).to(TYPES[c["x"]])}
    x = _values(g, c["M"], c["D"]).to(TYPES[c["x"]])
    w = (1 + 0.2 * torch.randn((c["D"],), generator=g, device="cuda")).to(TYPES[c["w"]])
    if c["op"] == "rms":
        r = (3 * _values(g, c["M"], c["D"])).to(TYPES[c["x"]]) if c["residual"] else None
        return {"case": c, "x": x, "w": w, "residual": r}
    dy = (1e-3 * torch.randn((c["M"], c["D"]), generator=g, device="cuda")).to(TYPES[c["x"]])
    dh = (1e-3 * torch.randn((c["M"], c["D"]), generator=g, device="cuda")).to(TYPES[c["x"]]) if c["dh"] else None
    rstd = torch.rsqrt(x.double().square().mean(1) + EPS).float()
    return {"case": c, "dy": dy, "h": x, "w": w, "rstd": rstd, "dh": dh}


# ---- the plain forms --------------------------------------------------------

def _amax(x, rows):
    """The largest |x| of each block of `rows` x 128."""
    m, k = x.shape
    p = torch.zeros((-(-m // rows) * rows, _blocks(k) * BLOCK), dtype=x.dtype, device=x.device)
    p[:m, :k] = x.abs()
    return p.view(p.shape[0] // rows, rows, _blocks(k), BLOCK).amax(dim=(1, 3))


def _spread_out(s, rows, m, k):
    """Each block's value at each of its elements."""
    return s.repeat_interleave(BLOCK, 1)[:, :k].repeat_interleave(rows, 0)[:m]


def _scale(amax, fp8, pow2):
    top = torch.full((), TOP[fp8], dtype=amax.dtype, device=amax.device)
    s = torch.clamp_min(amax / top, 2.0 ** -126)
    if pow2:
        m, e = torch.frexp(s)
        s = torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))
    return s


def _quantize(x, fp8, rows, pow2):
    x = x.float()
    s = _scale(_amax(x, rows), fp8, pow2)
    r = torch.ones_like(s) / s
    return (x * _spread_out(r, rows, *x.shape)).to(FP8[fp8]), s


def _product(s):
    c = s["case"]
    rows = BLOCK if c["sb"] == "tile" else 1
    a = s["a"].float() * _spread_out(s["sa"], 1, c["M"], c["K"])
    b = s["b"].float() * _spread_out(s["sb"], rows, c["N"], c["K"])
    return (a @ b.t()).to(TYPES[c["out"]])


def _quantized(s):
    c, x = s["case"], s["x"]
    rows = BLOCK if c["block"] == "tile" else 1
    q = _quantize(x, c["fp8"], rows, c["pow2"])
    if not c["transpose"]:
        return q
    return q + _quantize(x.t(), c["fp8"], rows, c["pow2"])


def _rms(s):
    x = s["x"]
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    f = h.float()
    rstd = torch.rsqrt(f.square().mean(1) + EPS)
    q, scale = _quantize(f * rstd[:, None] * s["w"].float(), "e4m3", 1, False)
    return q, scale, h, rstd


def _rms_backward(s):
    dy, h, rstd = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
    g = dy * s["w"].float()
    dx = rstd * (g - h * (rstd * rstd * (g * h).mean(1, keepdim=True)))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dx.to(s["h"].dtype), (dy * h * rstd).sum(0)


def _own(s):
    from software_pipelined_tiled_02_amd import binding
    c = s["case"]
    if c["op"] == "product":
        return binding.run_fp8(s["a"], s["sa"], s["b"], s["sb"], out_dtype=TYPES[c["out"]])
    if c["op"] == "quantize":
        return binding.quantize_fp8(s["x"], block=c["block"], fp8=c["fp8"], pow2=c["pow2"], transpose=c["transpose"])
    if c["op"] == "rms":
        return binding.rms_fp8(s["x"], s["w"], residual=s["residual"], eps=EPS)
    return binding.rms_backward(s["dy"], s["h"], s["w"], s["rstd"], dh=s["dh"])


def run(state):
    if own:
        return _own(state)
    return {"product": _product, "quantize": _quantized, "rms": _rms, "rms_backward": _rms_backward}[state["case"]["op"]](state)


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    c, size = case, {"bf16": 2, "f16": 2, "f32": 4}
    M = c["M"]
    if c["op"] == "product":
        N, K = c["N"], c["K"]
        scales = _blocks(K) * (M + (_blocks(N) if c["sb"] == "tile" else N))
        return {"bytes": M * K + N * K + 4 * scales + M * N * size[c["out"]], "flops": 2 * M * N * K}
    if c["op"] == "quantize":
        K, tile = c["K"], c["block"] == "tile"
        scales = _blocks(K) * (_blocks(M) if tile else M)
        if c["transpose"]:
            scales += _blocks(M) * (_blocks(K) if tile else K)
        return {"bytes": M * K * (size[c["x"]] + (2 if c["transpose"] else 1)) + 4 * scales, "flops": 2 * M * K}
    D = c["D"]
    if c["op"] == "rms":
        moved = size[c["x"]] * (3 if c["residual"] else 1) + 1
        return {"bytes": M * D * moved + 4 * M * _blocks(D) + 4 * M + D * size[c["w"]], "flops": 6 * M * D}
    moved = size[c["x"]] * (4 if c["dh"] else 3)
    return {"bytes": M * D * moved + 4 * M + D * (4 + size[c["w"]]), "flops": 9 * M * D}


# ---- the definitions in 64 bits ---------------------------------------------

def _exact_scales(x, fp8, rows, pow2):
    m, k = x.shape
    ki = torch.arange(k, device=x.device) // BLOCK
    mi = torch.arange(m, device=x.device) // rows
    by_k = torch.zeros((m, _blocks(k)), dtype=torch.float64, device=x.device).scatter_reduce_(
        1, ki.expand(m, k), x.abs(), "amax")
    s = torch.zeros((-(-m // rows), _blocks(k)), dtype=torch.float64, device=x.device).scatter_reduce_(
        0, mi[:, None].expand(m, _blocks(k)), by_k, "amax")
    s = (s / TOP[fp8]).clamp_min(2.0 ** -126)
    if pow2:
        s = torch.exp2(torch.ceil(torch.log2(s)))
    return s, s[mi][:, ki]


def _exact_quantize(x, fp8, rows, pow2, rounded):
    s, at = _exact_scales(x, fp8, rows, pow2)
    q = x / at
    return (q.to(FP8[fp8]).double() if rounded else q), s


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "product":
        ki = torch.arange(c["K"], device="cuda") // BLOCK
        ni = torch.arange(c["N"], device="cuda") // (BLOCK if c["sb"] == "tile" else 1)
        a = s["a"].double() * s["sa"].double()[:, ki]
        b = s["b"].double() * s["sb"].double()[ni][:, ki]
        return torch.mm(a, b.t())
    if c["op"] == "quantize":
        rows = BLOCK if c["block"] == "tile" else 1
        x = s["x"].double()
        q = _exact_quantize(x, c["fp8"], rows, c["pow2"], True)
        return q + _exact_quantize(x.t().contiguous(), c["fp8"], rows, c["pow2"], True) if c["transpose"] else q
    if c["op"] == "rms":
        h = s["x"].double()
        if s["residual"] is not None:
            h = h + s["residual"].double()
        f = h.to(s["x"].dtype).double()  # what the residual stream holds is what is normalised
        rstd = (f.square().sum(1) / c["D"] + EPS).pow(-0.5)
        # The values before their rounding to 8 bits: one next to a border may go to either side.
        q, scale = _exact_quantize(f * rstd[:, None] * s["w"].double(), "e4m3", 1, False, False)
        return q, scale, h, rstd
    dy, h, w, r = s["dy"].double(), s["h"].double(), s["w"].double(), s["rstd"].double()
    dot = (dy * w * h).sum(1) / c["D"]
    dx = (dy * w) * r[:, None] - h * (r ** 3 * dot)[:, None]
    if s["dh"] is not None:
        dx = dx + s["dh"].double()
    return dx, torch.mv((dy * h).t().contiguous(), r)
