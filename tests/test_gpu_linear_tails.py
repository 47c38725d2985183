"""The activations and their derivatives where the logistic function's or the
normal tail's value is under 2^-126 but the result is not: within R.ACT of the
value there too, and the derivative within R.ACT of its terms.  A result under 2^-126,
fp32's smallest normal number, may be 0."""
import pytest
import torch

from software_pipelined_tiled_02_amd import binding
from tests import linear_ref as R
from tests.linear_ref import assert_within

pytestmark = pytest.mark.gpu

NORMAL = 2.0 ** -126
LEAST = 2.0 ** -146            # a few roundings among fp32's subnormal numbers, whose step is 2^-149
BOTH = ("gelu", "gelu_tanh", "silu")


def arguments():
    """fp32 values, close to one another where the tails of the three leave the normal numbers, and the smallest and largest ones."""
    parts = [torch.linspace(a, b, 3001, dtype=torch.float64) for a, b in ((-140, 140), (-95, -84), (-14, -12), (-10.6, -9.4))]
    ends = torch.tensor([s * 2.0 ** e for s in (-1, 1) for e in (-120, -119, -118, -117, -60, -1, 0, 60, 119, 120, 126)], dtype=torch.float64)
    return torch.cat(parts + [ends]).float().cuda()


def held(got, ref, off, name):
    """Within `off` and bf16's half step where the result is a normal number."""
    here = ref.abs() >= NORMAL
    assert_within(got[here], ref[here], (off + R.half_step(ref.abs() + off, "bf16"))[here], name)
    assert bool(((got.double() - ref).abs()[~here] <= NORMAL).all()), name


@pytest.mark.parametrize("activation", BOTH)
def test_tails_of_activations(activation):
    z = arguments()
    n = z.numel()
    zero = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    ref = R.act(z.double(), activation)
    keep = ref.abs() <= torch.finfo(torch.bfloat16).max
    assert bool((ref.abs() < 2.0 ** -125).any()) and bool(keep.all())
    for tile in ("auto", "128x128"):
        c = binding.linear(zero(3, 8), zero(n, 8), bias=z, activation=activation, tile=tile)
        for row in c:
            held(row, ref, R.ACT * ref.abs() + LEAST, activation)


@pytest.mark.parametrize("activation", BOTH)
def test_tails_times_a_large_factor(activation):
    """H = act(G) U with U = 2^60: a lost tail would be seen from far."""
    z = arguments()
    ref = R.act(z.double(), activation) * 2.0 ** 60
    keep = (ref.abs() >= 2.0 ** -66) & (ref.abs() < 2.0 ** 127)
    zero = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    w = zero(z.numel(), 8)
    h = binding.gated(zero(2, 8), w, w, gate_bias=z, up_bias=torch.full_like(z, 2.0 ** 60), activation=activation)
    off = (R.ACT + R.U) * ref.abs() + 2.0 ** 60 * LEAST
    for row in h:
        assert_within(row[keep], ref[keep], (off + R.half_step(ref.abs() + off, "bf16"))[keep], activation)


@pytest.mark.parametrize("activation", BOTH)
def test_tails_of_derivatives(activation):
    """Every bf16 value up to 140 in size."""
    z = torch.arange(-32768, 32768, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    z = z[z.abs() <= 140][:, None]
    one = torch.ones((z.shape[0], 1), dtype=torch.bfloat16, device="cuda")
    dz, h = binding.gated_backward(one, one[:1], z, activation=activation, keep=True)
    ref, terms = R.slope(z.double(), activation)
    held(dz, ref, R.ACT * terms + LEAST, "derivative")
    ref = R.act(z.double(), activation)
    held(h, ref, R.ACT * ref.abs() + LEAST, "activation")
