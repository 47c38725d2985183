"""The feed-forward operators at the ends of what they take: more tiles than
CUs, long sums, rows far apart, and what the binding refuses."""
import pytest
import torch

from software_pipelined_tiled_02_amd import binding
from tests import linear_ref as R
from tests.linear_ref import FT, assert_within

pytestmark = pytest.mark.gpu
ALL = tuple(binding.LINEAR_TILES)


def rand(g, rows, cols, dtype="bf16", size=1.0):
    return (size * torch.randn((rows, cols), generator=g, device="cuda")).to(FT[dtype])


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# More tiles than one round of the CUs, for the large classes too; K of several
# K-tiles, not whole ones, from another one on in each XCD.
@pytest.mark.parametrize("dtype", ("bf16", "f16"))
@pytest.mark.parametrize("tile", ALL)
def test_more_tiles_than_cus(tile, dtype):
    M, N, K = (4400, 4168, 712) if tile in ("auto", "256x256", "128x256") else (1100, 2100, 712)
    g = gen(30)
    a, b, a2, b2 = rand(g, M, K, dtype), rand(g, N, K, dtype, K ** -0.5), rand(g, M, K, dtype), rand(g, N, K, dtype, K ** -0.5)
    r = rand(g, M, N, dtype)
    c, z = binding.linear(a, b, activation="silu", residual=r, keep=True, tile=tile)
    want, off, zwant, zoff = R.linear(a.double(), b.double().t(), dtype, activation="silu", residual=r.double())
    assert_within(c, want, off, "c")
    assert_within(z, zwant, zoff, "z")
    pair = (a2.double(), b2.double().t())
    want, off = R.linear(a.double(), b.double().t(), dtype, pair=pair)[:2]
    assert_within(binding.linear(a, b, pair=(a2, b2), tile=tile), want, off, "RC pair")
    rr = b.t().contiguous(), b2.t().contiguous()
    assert_within(binding.linear(a, rr[0], layout="RR", pair=(a2, rr[1]), tile=tile), want, off, "RR pair")
    if tile != "16x16":
        for v, (want, off), name in zip(binding.gated(a, b, b2, keep=True, tile=tile),
                                        R.gated(a.double(), b.double(), b2.double(), dtype, "silu"), "hgu"):
            assert_within(v, want, off, name)
    up = rand(g, M, N, dtype)
    for v, (want, off), name in zip(binding.gated_backward(a, rr[0], r, up, keep=True, tile=tile),
                                    R.gated_backward(a.double(), rr[0].double(), r.double(), up.double(), dtype, "silu"), ("dg", "du", "h")):
        assert_within(v, want, off, name)


@pytest.mark.parametrize("tile", ALL[:8])
def test_weight_gradient_of_more_tiles_than_cus(tile):
    M, N, K = (712, 4400, 4168) if tile in ("auto", "256x256", "128x256") else (712, 1100, 2100)
    g = gen(31)
    dc, a = rand(g, M, N), rand(g, M, K)
    dw, off, db, db_off = R.weight_gradient(dc.double(), a.double())
    got, sums = binding.weight_gradient(dc, a, bias=True, tile=tile)
    assert_within(got, dw, off, "dw")
    assert_within(sums, db, db_off, "db")


@pytest.mark.parametrize("tile", ALL)
def test_long_sums(tile):
    """K of 130 K-tiles and a part of one; K-tiles by turns of 4 and 8 waves."""
    M, N, K = 70, 130, 8324
    g = gen(32)
    for dtype in ("bf16", "f16"):
        a, b = rand(g, M, K, dtype), rand(g, N, K, dtype, K ** -0.5)
        want, off = R.linear(a.double(), b.double().t(), dtype)[:2]
        assert_within(binding.linear(a, b, tile=tile), want, off, "RC")
        assert_within(binding.linear(a, b.t().contiguous(), layout="RR", tile=tile), want, off, "RR")
        if tile not in ("16x32", "16x16"):
            dw, off, db, db_off = R.weight_gradient(a.double().t(), b.double().t())
            got, sums = binding.weight_gradient(a.t().contiguous(), b.t().contiguous(), bias=True, tile=tile)
            assert_within(got, dw, off, "dw")
            assert_within(sums, db, db_off, "db")


def far(t, ld):
    """t in rows `ld` apart, in a buffer that is not filled."""
    rows, cols = t.shape
    flat = torch.empty((rows - 1) * ld + cols, dtype=t.dtype, device="cuda")
    return flat.as_strided((rows, cols), (ld, 1)).copy_(t)


@pytest.mark.parametrize("rows_far", ("inputs", "outputs"))
def test_rows_beyond_32_bits(rows_far):
    """Matrices whose last rows lie past 2^32 bytes: of the input, the weight, what is read beside the sums, and results."""
    M, N, K, ld = 1300, 1270, 72, 2 ** 21 + 8                # 1270 rows of 4 MB: 5.3e9 bytes
    g = gen(33)
    a, b, dc = rand(g, M, K), rand(g, N, K, size=K ** -0.5), rand(g, M, N)
    b2, r = rand(g, N, K, size=K ** -0.5), rand(g, M, N)
    if rows_far == "inputs":
        for x, w, add in ((far(a, ld), b, r), (a, far(b, ld), r), (a, b, far(r, ld))):
            c = binding.linear(x, w, residual=add)
            assert_within(c, *R.linear(a.double(), b.double().t(), "bf16", residual=r.double())[:2], "c")
        (h, hoff), _, _ = R.gated(a.double(), b.double(), b2.double(), "bf16", "silu")
        assert_within(binding.gated(a, b, far(b2, ld)), h, hoff, "h")
        want = R.gated_backward(a.double(), b.double().t(), r.double(), dc.double(), "bf16", "silu")
        for gate, up in ((far(r, ld), dc), (r, far(dc, ld))):
            for v, (ref, off) in zip(binding.gated_backward(a, b.t().contiguous(), gate, up), want):
                assert_within(v, ref, off, "dg, du")
        dw, off = R.weight_gradient(dc.double(), a.double())[:2]
        for x, y in ((far(dc, ld), a), (dc, far(a, ld))):
            assert_within(binding.weight_gradient(x, y), dw, off, "dw")
        # the weight's rows along the sums of the layer's input's gradient
        want, off = R.linear(dc.double(), b.double(), "bf16")[:2]
        assert_within(binding.linear(dc, far(b, ld), layout="RR"), want, off, "RR")
    else:
        out = far(torch.zeros_like(r), ld)
        assert binding.linear(a, b, out=out) is out
        assert_within(out, *R.linear(a.double(), b.double().t(), "bf16")[:2], "c")
        dw = far(torch.zeros((N, K), device="cuda"), ld // 2)
        binding.weight_gradient(dc, a, out=dw)
        assert_within(dw, *R.weight_gradient(dc.double(), a.double())[:2], "dw")
        binding.gated(a, b, b2, out=out)
        assert_within(out, *R.gated(a.double(), b.double(), b2.double(), "bf16", "silu")[0], "h")


def test_many_rows():
    """More rows than 16 bits count, of one column and of one value."""
    g = gen(34)
    M = 140000
    a, b = rand(g, M, 8), rand(g, 3, 8)
    assert_within(binding.linear(a, b), *R.linear(a.double(), b.double().t(), "bf16")[:2], "c")
    assert_within(binding.linear(b, a), *R.linear(b.double(), a.double().t(), "bf16")[:2], "c, many columns")
    dw, off, db, db_off = R.weight_gradient(a.double(), a[:, :1].double())
    got, sums = binding.weight_gradient(a, a[:, :1], bias=True)
    assert_within(got, dw, off, "dw")
    assert_within(sums, db, db_off, "db")


def test_results_do_not_change_from_run_to_run():
    g = gen(35)
    a, b, dc = rand(g, 333, 1000), rand(g, 700, 1000), rand(g, 333, 700)
    first = binding.linear(a, b, activation="gelu"), *binding.weight_gradient(dc, a, bias=True)
    for _ in range(20):
        again = binding.linear(a, b, activation="gelu"), *binding.weight_gradient(dc, a, bias=True)
        assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_refusals():
    """Before anything is enqueued."""
    e = lambda *s, t=torch.bfloat16: torch.ones(s, dtype=t, device="cuda")  # noqa: E731
    x, w, r = e(4, 64), e(32, 64), e(4, 32)
    L, G, D, W = binding.linear, binding.gated, binding.gated_backward, binding.weight_gradient
    bad = [lambda: L(x, e(32, 65)), lambda: L(x, w, layout="RR"), lambda: L(x, e(32, 64, t=torch.float16)), lambda: L(x, w.float()),
           lambda: L(x, w.cpu()), lambda: L(x.t(), w), lambda: L(x[:, ::2], w[:, ::2]), lambda: L(x[0], w), lambda: L(x, w, bias=e(31)),
           lambda: L(x, w, bias=e(32, t=torch.float16)), lambda: L(x, w, bias=e(32, 1)), lambda: L(x, w, residual=e(4, 33)),
           lambda: L(x, w, residual=e(1, 32)), lambda: L(x, w, residual=r[:1].expand(4, 32)), lambda: L(x, w, residual=r.float()),
           lambda: L(x, w, pair=(e(4, 63), e(32, 63))), lambda: L(x, w, pair=(x, e(31, 64))), lambda: L(x, w, out=e(4, 33)),
           lambda: L(x, w, out=e(4, 32, t=torch.float32)), lambda: L(x, w, out=e(32, 4).t()), lambda: L(x, w, out=r[:1].expand(4, 32)),
           lambda: L(e(4, 64, t=torch.float32), w.float()),
           lambda: G(x, w, e(31, 64)), lambda: G(x, w, e(32, 63)), lambda: G(x, w, w.half()), lambda: G(x, w, w, gate_bias=e(33)),
           lambda: G(x, w, w, gate_bias=e(32), up_bias=e(32, t=torch.float32)), lambda: G(x, w, w, out=e(4, 31)), lambda: G(x, w, None),
           lambda: D(x, w, r), lambda: D(x, e(64, 32), e(4, 31)), lambda: D(x, e(64, 32), r, e(3, 32)), lambda: D(x, e(64, 32), r.half()),
           lambda: D(x, e(64, 32), None),
           lambda: W(r, e(5, 64)), lambda: W(r, x.half()), lambda: W(r, x, accumulate=True), lambda: W(r, x, out=e(32, 64)),
           lambda: W(r, x, out=e(32, 63, t=torch.float32)), lambda: W(r, x, bias_out=e(32)), lambda: W(r, x, bias_out=e(31, t=torch.float32)),
           lambda: W(r, x, out=e(32, 64, t=torch.float32), bias=True, accumulate=True), lambda: W(r, e(4, 0), bias=True)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail("call %d was not refused" % i)
    with pytest.raises(binding.GemmError) as err:
        G(x, w, w, tile="16x16")
    assert err.value.status == binding.GEMM_ERR_UNSUPPORTED
    with pytest.raises(binding.GemmError) as err:
        W(r, x, tile="16x32")
    assert err.value.status == binding.GEMM_ERR_UNSUPPORTED
    assert bool((L(x, w) == 64).all())                         # and the next call is fine


def test_results_over_what_is_read():
    """Refused, but for a residual's own place; columns beside one another do not overlap."""
    g = gen(36)
    buf = rand(g, 96, 256)
    a, w, r = buf[:64, :64], rand(g, 64, 64), rand(g, 64, 64)
    L, G, W = binding.linear, binding.gated, binding.weight_gradient
    other = rand(g, 64, 64)
    floats = torch.zeros((64, 65), device="cuda")
    for call in (lambda: L(a, w, out=a), lambda: L(a, w, out=w), lambda: L(a, w, out=buf[32:, :64]), lambda: L(a, w, out=buf[:64, 63:127]),
                 lambda: L(a, w, out=buf[:64, 1:65]), lambda: L(other, w, pair=(a, r), out=buf[5:69, :64]),
                 lambda: L(other, w, residual=a, out=buf[1:65, :64]), lambda: L(other, w, residual=a, out=buf.view(192, 128)[:64, :64]),
                 lambda: L(other, w, bias=buf[70, 3:67], out=buf[20:84, :64]), lambda: G(a, w, r, out=a), lambda: G(other, w, r, out=r),
                 lambda: G(other, w, r, up_bias=buf[0, :64], out=a),
                 lambda: W(other.float()[:1].view(torch.bfloat16)[:, :64], a, out=floats[:, :64], bias_out=floats[3, :64]),
                 lambda: W(floats.view(torch.bfloat16)[:, :64], a, out=floats[:, :64])):
        with pytest.raises(ValueError):
            call()
    want = L(a, w, residual=r)
    got = buf[:64, 64:128]
    assert L(a, w, residual=r, out=got) is got and torch.equal(got, want)
    got = buf[:64, 128:192].copy_(r)
    assert torch.equal(L(a, w, residual=got, out=got), want)
    assert torch.equal(G(a, w, r, out=buf[3:67, 192:]), G(a, w, r))
