"""The feed-forward operators beside torch's autograd: their results carry no
gradient, what they write in place is noticed, and a torch.autograd.Function of
them is differentiated."""
import pytest
import torch

from software_pipelined_tiled_02_amd import binding
from tests import linear_ref as R

pytestmark = pytest.mark.gpu


def rand(*shape, seed=0, size=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (size * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def test_results_carry_no_gradient():
    x, w = rand(5, 64).requires_grad_(), rand(32, 64, seed=1).requires_grad_()
    z = rand(5, 32, seed=2).requires_grad_()
    results = [binding.linear(x, w), *binding.gated(x, w, w, keep=True), *binding.gated_backward(x, w.t().contiguous(), z, z),
               *binding.weight_gradient(z, x, bias=True)]
    assert not any(t.requires_grad for t in results)


def test_what_is_written_in_place_is_noticed():
    """A tensor that autograd has kept and an operator then writes: backward refuses, as behind torch's own operators in place."""
    x, w = rand(5, 64), rand(32, 64, seed=1)

    def writes(call, kept):
        s = torch.ones((), device="cuda", requires_grad=True)
        y = s * kept                                          # keeps `kept`
        before = kept._version
        call(kept)
        assert kept._version > before
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()

    r = rand(5, 32, seed=2)
    writes(lambda t: binding.linear(x, w, residual=t, out=t), r)
    writes(lambda t: binding.linear(x, w, out=t), r)
    writes(lambda t: binding.gated(x, w, w, out=t), r)
    writes(lambda t: binding.weight_gradient(r, x, out=t, accumulate=True), torch.zeros((32, 64), device="cuda"))
    writes(lambda t: binding.weight_gradient(r, x, bias_out=t), torch.zeros(32, device="cuda"))
    writes(lambda t: binding.linear(x, w, residual=t[:, :32], out=t[:, :32]), rand(5, 40, seed=3))        # of a view, its base's
    with torch.inference_mode():                              # such tensors count no versions
        t = rand(5, 32, seed=4)
    want = binding.linear(x, w, residual=t.clone())
    assert torch.equal(binding.linear(x, w, residual=t, out=t), want)
    refused = r._version
    with pytest.raises(ValueError):
        binding.linear(x, w, residual=r[:, :31], out=r)
    assert r._version == refused


class Block(torch.autograd.Function):
    """y = x + (silu(x gate^T) * (x up^T)) down^T"""

    @staticmethod
    def forward(ctx, x, gate, up, down):
        h, g, u = binding.gated(x, gate, up, keep=True)
        ctx.save_for_backward(x, gate, up, down, g, u)
        return binding.linear(h, down, residual=x)

    @staticmethod
    def backward(ctx, dy):
        x, gate, up, down, g, u = ctx.saved_tensors
        dg, du, h = binding.gated_backward(dy, down, g, u, keep=True)
        dx = binding.linear(dg, gate, layout="RR", pair=(du, up), residual=dy)
        return (dx, *(binding.weight_gradient(d, t).to(x.dtype) for d, t in ((dg, x), (du, x), (dy, h))))


def test_as_an_autograd_function():
    D, F = 136, 200
    leaves = [t.requires_grad_() for t in (rand(70, D), rand(F, D, seed=1, size=D ** -0.5), rand(F, D, seed=2, size=D ** -0.5),
                                           rand(D, F, seed=3, size=F ** -0.5))]
    dy = rand(70, D, seed=4)
    Block.apply(*leaves).backward(dy)
    exact = [t.detach().double().requires_grad_() for t in leaves]
    x, gate, up, down = exact
    (x + (R.act(x @ gate.t(), "silu") * (x @ up.t())) @ down.t()).backward(dy.double())
    for got, want in zip(leaves, exact):
        # g or u, dg or du, and the result are rounded: three half steps of 2^-8, not all one way
        assert float((got.grad.double() - want.grad).norm()) < 2.0 ** -6 * float(want.grad.norm())
