"""The feed-forward operators with one tensor in several places, with one bias of
two, and with subnormal values in their factors."""
import pytest
import torch

from software_pipelined_tiled_02_amd import binding
from tests import linear_ref as R
from tests.linear_ref import FT, assert_within

pytestmark = pytest.mark.gpu
SIZES = ((1, 72, 40), (70, 70, 70), (300, 264, 200), (513, 129, 64))


def rand(g, rows, cols, dtype, size=1.0):
    return (size * torch.randn((rows, cols), generator=g, device="cuda")).to(FT[dtype])


@pytest.mark.parametrize("dtype", ("bf16", "f16"))
@pytest.mark.parametrize("M,N,K", SIZES)
def test_one_tensor_in_several_places(M, N, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(50)
    a, w, r = rand(g, M, K, dtype), rand(g, N, K, dtype, K ** -0.5), rand(g, M, N, dtype)
    d = lambda t: t.double()  # noqa: E731
    for layout, b in (("RC", w), ("RR", w.t().contiguous())):
        ref = d(w).t()
        c = binding.linear(a, b, layout=layout, pair=(a, b), residual=r)
        assert_within(c, *R.linear(d(a), ref, dtype, residual=d(r), pair=(d(a), ref))[:2], "pair")
    for v, (want, off) in zip(binding.gated(a, w, w, keep=True), R.gated(d(a), d(w), d(w), dtype, "silu")):
        assert_within(v, want, off, "gated")
    x = rand(g, M, N, dtype)
    wd = rand(g, N, N, dtype, N ** -0.5)
    for v, (want, off) in zip(binding.gated_backward(x, wd, x, x, keep=True), R.gated_backward(d(x), d(wd), d(x), d(x), dtype, "silu")):
        assert_within(v, want, off, "gated_backward")
    dw, off, db, db_off = R.weight_gradient(d(a), d(a))
    got, sums = binding.weight_gradient(a, a, bias=True)
    assert_within(got, dw, off, "dw")
    assert_within(sums, db, db_off, "db")
    square = rand(g, K, K, dtype, K ** -0.5)
    assert_within(binding.linear(square, square, residual=square), *R.linear(d(square), d(square).t(), dtype, residual=d(square))[:2], "square")


@pytest.mark.parametrize("kind", ("f32", "own"))
@pytest.mark.parametrize("which", ("gate", "up"))
def test_one_bias_of_two(which, kind):
    g = torch.Generator(device="cuda").manual_seed(51)
    x, wg, wu = rand(g, 70, 64, "bf16"), rand(g, 130, 64, "bf16", 0.1), rand(g, 130, 64, "bf16", 0.1)
    b = torch.randn(130, generator=g, device="cuda")
    b = b if kind == "f32" else b.bfloat16()
    got = binding.gated(x, wg, wu, keep=True, **{which + "_bias": b})
    ref = R.gated(x.double(), wg.double(), wu.double(), "bf16", "silu", **{"b" + which[0]: b.double()})
    for v, (want, off) in zip(got, ref):
        assert_within(v, want, off, which)


@pytest.mark.parametrize("dtype,small,large", (("bf16", 2.0 ** -130, 2.0 ** 100), ("f16", 2.0 ** -20, 2.0 ** 10)))
@pytest.mark.parametrize("tile", binding.LINEAR_TILES)
def test_subnormal_factors_count(tile, dtype, small, large):
    """Numbers below the type's smallest normal one, times large ones."""
    g = torch.Generator(device="cuda").manual_seed(52)
    whole = lambda *s: torch.randint(-7, 8, s, generator=g, device="cuda").double()  # noqa: E731
    a, b = whole(70, 72), whole(40, 72)
    low, high = (a * small).to(FT[dtype]), (b * large).to(FT[dtype])
    assert torch.equal(low.double(), a * small) and torch.equal(high.double(), b * large)
    want = (a @ b.t() * (small * large)).to(FT[dtype])
    assert torch.equal(binding.linear(low, high, tile=tile), want)
    assert torch.equal(binding.linear(high, low, tile=tile), want.t())
    if tile not in ("16x32", "16x16"):
        dw, db = binding.weight_gradient(low.t().contiguous(), high.t().contiguous(), bias=True, tile=tile)
        assert torch.equal(dw.double(), a @ b.t() * (small * large))
        assert torch.equal(db.double(), (a * small).sum(1).float().double())
