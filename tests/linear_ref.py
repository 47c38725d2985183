"""The feed-forward operators from their definitions, in 64 bits (torch, on
the CPU or the GPU), and the error bounds the tests hold the kernels to.

Bounds.  Products of two 16-bit values are exact in fp32.  A sum of n products
in fp32, in any order and grouping, is off by less than n v sum |a b| with v =
2^-23 (an addition in the matrix core may truncate); n v < 2^-8 throughout, so
second-order terms are covered by the factor 1.01.  An activation as computed is
off by less than ACT of its value; its derivative by less than ACT of its two
terms' sizes (they may cancel): the argument of the exponential, up to 126 in
size, has two roundings of 2^-24, which make up to 2^-16.5 of its value, the
rest is below 2^-17.  A factor below 2^-126 (the logistic function's or the normal
tail's value) is a subnormal and may be flushed to 0: the product with z is off by
up to |z| 2^-126 then, and the derivative by that times q' + 1 (`flushed`, for |z| up to
128, past which both are taken at 128).  |act'| <= 1.13, so an error of the argument counts 1.13 times.  fp32 operations behind that are
off by 2^-24 each, and the last rounding by half a step: eps / 2 of the value, or of
the smallest normal one.
"""
import math

import torch

FT = {"bf16": torch.bfloat16, "f16": torch.float16}
V, U = 2.0 ** -23, 2.0 ** -24
ACT = 2.0 ** -16
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")
_C = 2 * math.sqrt(2 / math.pi)


def _logistic_of(z, name):
    """(q, q') with act(z) = z s(q), s the logistic function."""
    if name == "silu":
        return z, torch.ones_like(z)
    return _C * (z + 0.044715 * z ** 3), _C * (1 + 3 * 0.044715 * z * z)


def act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), z)       # (a NaN stays)
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    return z * torch.special.expit(_logistic_of(z, name)[0])


def slope(z, name):
    """(act'(z), the sizes of its terms together)"""
    if name == "none":
        one = torch.ones_like(z)
        return one, one
    if name == "relu":
        d = torch.where(z > 0, torch.ones_like(z), torch.zeros_like(z))
        return torch.where(z == z, d, z), d
    if name == "gelu":
        p, q = 0.5 * torch.special.erfc(-z / math.sqrt(2)), z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    else:
        x, dx = _logistic_of(z, name)
        p = torch.special.expit(x)
        q = z * p * torch.special.expit(-x) * dx
    return p + q, p.abs() + q.abs()


def flushed(z, of_slope=False):
    """What a factor of act(z), or of act'(z), that is flushed to 0 makes at most."""
    z = z.abs().clamp_max(128.0).nan_to_num(128.0)
    return 2.0 ** -126 * (1 + z * (1 if not of_slope else 1.6 + 0.22 * z * z))


def half_step(x, dtype):
    """Half a step of the type at values up to |x|."""
    f = torch.finfo(FT[dtype])
    return torch.clamp_min(x.abs(), f.smallest_normal) * (f.eps / 2)


def sums(a, b):
    """(a b, how far a sum in fp32 may be off); a: M x K, b: K x N, in 64 bits."""
    return a @ b, 1.01 * V * a.shape[1] * (a.abs() @ b.abs())


def linear(a, b, dtype, bias=None, activation="none", residual=None, pair=None):
    """(c, its bound, z, its bound); a: M x K, b: K x N, all in 64 bits."""
    z, off = sums(a, b)
    if pair is not None:
        z2, off2 = sums(*pair)
        z, off = z + z2, off + off2 + V * (z.abs() + z2.abs())
    if bias is not None:
        z = z + bias
        off = off + U * z.abs()
    y = act(z, activation)
    far = 1.13 * off + ACT * y.abs()
    if residual is not None:
        y = y + residual
        far = far + U * y.abs()
    return y, far + half_step(y.abs() + far, dtype), z, off + half_step(z.abs() + off, dtype)


def gated(x, wg, wu, dtype, activation, bg=None, bu=None):
    """((h, bound), (g, bound), (u, bound)); wg, wu: N x K."""
    one = [linear(x, w.t(), dtype, b) for w, b in ((wg, bg), (wu, bu))]
    (g, g_off), (u, u_off) = ((z, sums(x, w.t())[1] + U * z.abs()) for (_, _, z, _), w in zip(one, (wg, wu)))
    a = act(g, activation)
    a_off = 1.13 * g_off + ACT * a.abs()
    h = a * u
    off = a_off * (u.abs() + u_off) + a.abs() * u_off + U * h.abs()
    return (h, off + half_step(h.abs() + off, dtype)), one[0][2:], one[1][2:]


def gated_backward(dy, w, g, u, dtype, activation):
    """[(dg, bound), (du, bound), (h, bound)]; w: K x N; u may be None (then without du)."""
    dh, off = sums(dy, w)
    a, (d, terms) = act(g, activation), slope(g, activation)
    a_off, d_off = ACT * a.abs(), ACT * terms
    s = torch.ones_like(g) if u is None else u
    out = [(dh * s * d, s.abs() * (off * d.abs() + (dh.abs() + off) * d_off)), (dh * a, off * a.abs() + (dh.abs() + off) * a_off),
           (a * s, a_off * s.abs())]
    if u is None:
        del out[1]
    out = [(v, e + 2 * U * (v.abs() + e)) for v, e in out]
    return [(v, e + half_step(v.abs() + e, dtype)) for v, e in out]


def weight_gradient(dc, a):
    """(dw, bound, db, bound)"""
    dw, off = sums(dc.t(), a)
    return dw, off, dc.sum(0), 1.01 * V * dc.shape[0] * dc.abs().sum(0)


def assert_within(got, ref, bound, what):
    got, ref = got.double(), ref.to(got.device)
    bound = bound.to(got.device)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    wrong = ~((got - ref).abs() <= bound)
    if bool(wrong.any()):
        i = int(wrong.flatten().to(torch.uint8).argmax())
        raise AssertionError("%s: %d of %d values off, the first at %d: %r, not %r (bound %g)" % (
            what, int(wrong.sum()), wrong.numel(), i, float(got.flatten()[i]), float(ref.flatten()[i]), float(bound.flatten()[i])))


def place(t, ld, offset=0, device="cuda"):
    """t with rows `ld` apart from element `offset` of a buffer of NaNs that ends with the last row's last value."""
    rows, cols = t.shape
    flat = torch.full((max(1, offset + (rows - 1) * ld + cols),), float("nan"), dtype=t.dtype, device=device)
    view = flat[offset:].as_strided((rows, cols), (ld, 1))
    return view.copy_(t)
