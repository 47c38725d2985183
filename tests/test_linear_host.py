"""The feed-forward operators on the CPU: the 64-bit reference against central
differences, the plan, and every refusal of the C entry points and of the
binding (all of them before any HIP call)."""
import pytest
import torch

from software_pipelined_tiled_02_amd import binding
from tests import linear_ref as R
from tests.test_fp8_host import FAKE

BAD, ALIGN, UNSUP, OK = (binding.GEMM_ERR_INVALID_ARG, binding.GEMM_ERR_ALIGNMENT, binding.GEMM_ERR_UNSUPPORTED,
                         binding.GEMM_OK)
H, P = FAKE.h, 4096        # a handle and an aligned address; refused calls never use them


# ---- the reference ----------------------------------------------------------

@pytest.mark.parametrize("activation", R.ACTIVATIONS)
def test_slope_is_the_activations_derivative(activation):
    z = torch.linspace(-9, 9, 4001, dtype=torch.float64)
    z = z[z.abs() > 1e-3]
    step = 1e-5        # truncation ~ step^2, rounding ~ 1e-16 * |act| / step: below 1e-9
    d = (R.act(z + step, activation) - R.act(z - step, activation)) / (2 * step)
    s, terms = R.slope(z, activation)
    assert float((d - s).abs().max()) < 1e-8 and bool((terms >= s.abs() - 1e-12).all())


def test_activations_are_torchs():
    z = torch.linspace(-9, 9, 1001, dtype=torch.float64)
    f = torch.nn.functional
    for name, want in (("relu", f.relu(z)), ("gelu", f.gelu(z)), ("gelu_tanh", f.gelu(z, approximate="tanh")), ("silu", f.silu(z))):
        assert float((R.act(z, name) - want).abs().max()) < 1e-13, name


@pytest.mark.parametrize("activation", ("silu", "gelu"))
def test_the_blocks_backward_is_its_derivative(activation):
    """h, g, u = gated(x); y = h wd^T + x: the gradients as the operators form
    them, against central differences, in 64 bits without roundings."""
    g = torch.Generator().manual_seed(0)
    n = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    M, D, F = 3, 5, 7
    x, wg, wu, wd, dy, bg = n(M, D), n(F, D), n(F, D), n(D, F), n(M, D), n(F)

    def forward(x, wg, wu, wd, bg):
        return ((R.act(x @ wg.t() + bg, activation) * (x @ wu.t())) @ wd.t() + x)

    gg, u = x @ wg.t() + bg, x @ wu.t()
    (dg, _), (du, _), (h, _) = R.gated_backward(dy, wd, gg, u, "bf16", activation)
    dx = R.linear(dg, wg, "bf16", pair=(du, wu), residual=dy)[0]
    dwg, _, dbg, _ = R.weight_gradient(dg, x)
    grads = {"x": dx, "wg": dwg, "wu": R.weight_gradient(du, x)[0], "wd": R.weight_gradient(dy, h)[0], "bg": dbg}
    args = dict(x=x, wg=wg, wu=wu, wd=wd, bg=bg)
    step = 1e-5
    for name, grad in grads.items():
        for i in range(0, grad.numel(), 3):
            d = torch.zeros_like(args[name]).flatten()
            d[i] = step
            d = d.view_as(args[name])
            up, down = (float((forward(**{**args, name: args[name] + s * d}) * dy).sum()) for s in (1, -1))
            assert abs((up - down) / (2 * step) - float(grad.flatten()[i])) < 1e-6, (name, i)


# ---- the plan ----------------------------------------------------------------

def q(form, M, N, K, **kw):
    return binding.gemm_query_linear(form, M, N, K, check=False, **kw)


def test_plan():
    for form in binding.LINEAR_FORMS:
        for M, N, K in ((1, 4096, 4096), (64, 8192, 8192), (500, 4104, 4100), (8192, 8192, 8200), (0, 16, 16), (16, 0, 16), (16, 16, 0),
                        (8192, 1000, 24), (7, 100000, 3)):
            for r16 in (True, False):
                rc, info = q(form, M, N, K, rows16=r16)
                assert rc == OK and info["rows16"] == int(r16)
                rows, cols, depth = (N, K, M) if form == "weight_gradient" else (M, N, K)
                want = -(-rows // info["block_m"]) * -(-cols // info["block_n"]) if rows and cols else 0
                assert info["grid"] == want and info["k_tiles"] == -(-depth // 64), (form, M, N, K, info)
    assert q("linear_rc", 8192, 8192, 8200)[1]["tile"] == binding.LINEAR_TILES["256x256"]


def test_plan_of_a_great_many_tiles():
    """The smallest classes would take more threads than a launch may have: others do it."""
    big = 2 ** 31 - 1024
    for form, M, N, K in (("linear_rc", 1, big, 64), ("linear_rr", big, 1, 64), ("gated", 3, big // 2, 64), ("weight_gradient", 2, big, 1)):
        for r16 in (True, False):
            rc, info = q(form, M, N, K, rows16=r16)
            assert rc == OK and info["grid"] * info["threads"] < 2 ** 32, (form, info)
    assert q("linear_rc", 1, big, 64, tile="16x16")[0] == UNSUP and q("linear_rc", big, big, 64)[0] == UNSUP


def test_query_refusals():
    assert q(5, 1, 1, 1)[0] == BAD and q(-1, 1, 1, 1)[0] == BAD
    for bad in (dict(dtype="f32"), dict(dtype="i8"), dict(rows16=2), dict(tile=99), dict(tile=-2)):
        assert q("gated", 1, 1, 1, **bad)[0] == BAD, bad
    assert q("gated", -1, 1, 1)[0] == BAD and q("gated", 1, -1, 1)[0] == BAD and q("gated", 1, 1, -1)[0] == BAD
    assert q("linear_rc", 2 ** 31, 1, 1)[0] == UNSUP and q("linear_rc", 1, 2 ** 31, 1)[0] == UNSUP
    assert q("linear_rc", 1, 1, 2 ** 31)[0] == UNSUP
    assert q("linear_rc", 2 ** 30, 2 ** 30, 1)[0] == UNSUP                      # 2^32 threads and more
    assert binding._lib().gemm_query_linear(0, 1, 1, 1, binding.GEMM_BF16, 1, -1, None) == BAD


# ---- refusals of the calls ---------------------------------------------------

def call(fn, args, kw):
    unknown = set(kw) - set(args)
    assert not unknown, unknown
    return fn(H, *{**args, **kw}.values(), stream=0, check=False)


def linear(**kw):
    return call(binding.gemm_linear, dict(M=64, N=64, K=64, dtype="bf16", layout="RC", act="none", bt="f32", tile="auto", A=P, lda=64, B=P,
                                          ldb=64, A2=P, lda2=64, B2=P, ldb2=64, bias=P, R=P, ldr=64, Z=P, ldz=64, C=P, ldc=64), kw)


def gated(**kw):
    return call(binding.gemm_gated, dict(M=64, N=64, K=64, dtype="f16", act="silu", bt="f16", tile="auto", X=P, ldx=64, WG=P, ldwg=64, WU=P,
                                         ldwu=64, BG=P, BU=P, G=P, ldg=64, U=P, ldu=64, Hh=P, ldh=64), kw)


def backward(**kw):
    return call(binding.gemm_gated_backward, dict(M=64, N=64, K=64, dtype="bf16", act="silu", tile="auto", DY=P, lddy=64, W=P, ldw=64, G=P,
                                                  ldg=64, U=P, ldu=64, DG=P, lddg=64, DU=P, lddu=64, Hh=P, ldh=64), kw)


def weight(**kw):
    return call(binding.gemm_weight_gradient, dict(M=64, N=64, K=64, dtype="bf16", acc=0, tile="auto", DC=P, lddc=64, A=P, lda=64, DW=P,
                                                   lddw=64, DB=P), kw)


FACTORS = ((linear, ("A", "B", "A2", "B2"), ("lda", "ldb", "lda2", "ldb2")), (gated, ("X", "WG", "WU"), ("ldx", "ldwg", "ldwu")),
           (backward, ("DY", "W"), ("lddy", "ldw")), (weight, ("DC", "A"), ("lddc", "lda")))
OTHERS = ((linear, ("R", "Z", "C"), ("ldr", "ldz", "ldc"), ("C",)), (gated, ("G", "U", "Hh"), ("ldg", "ldu", "ldh"), ("Hh",)),
          (backward, ("G", "U", "DG", "DU", "Hh"), ("ldg", "ldu", "lddg", "lddu", "ldh"), ("G", "DG")), (weight, ("DW",), ("lddw",), ("DW",)))


def test_refusals_of_every_operator():
    for fn, ps, lds in FACTORS:
        for bad in (dict(dtype="f32"), dict(dtype="i8"), dict(dtype=7), dict(M=-1), dict(N=-1), dict(K=-1), dict(tile=99), dict(tile=-2)):
            assert fn(**bad) == BAD, (fn, bad)
        for big in ("M", "N", "K"):
            assert fn(**{big: 2 ** 31 - 512}) == UNSUP, (fn, big)
        for p in ps:
            assert fn(**{p: P + 1}) == ALIGN, p
        for ld in lds:
            assert fn(**{ld: 63}) == BAD and fn(**{ld: -64}) == BAD, ld
            assert fn(**{ld: 2 ** 40}) == UNSUP, ld
        if fn is not linear:
            for p in ps:
                assert fn(**{p: None}) == BAD, p
    for fn, ps, lds, needed in OTHERS:
        size = 4 if fn is weight else 2
        for p in ps:
            assert fn(**{p: P + size - 1}) == ALIGN, p
        for p in needed:
            assert fn(**{p: None}) == BAD, p
        for ld in lds:
            assert fn(**{ld: 63}) == BAD, ld
    for fn in (linear, gated, backward):
        assert fn(act=-1) == BAD and fn(act=5) == BAD


def test_strides_at_the_border_of_the_offsets():
    """256 rows of a factor with K inside, or 64 of K, whether they are there or not, span less than 2^31 bytes."""
    lim = 2 ** 31 - 1024
    assert linear(M=300, lda=lim // 512 + 1) == UNSUP and linear(M=2, lda=lim // 4 + 1) == UNSUP
    assert linear(layout="RR", ldb=lim // 128 + 1) == UNSUP and linear(layout="RR", K=2, lda=64, ldb=lim // 128 + 1) == UNSUP
    assert weight(lddc=lim // 128 + 1) == UNSUP and backward(ldw=lim // 128 + 1) == UNSUP
    assert gated(N=256, ldg=256, ldu=256, ldh=256, ldwu=lim // 512 + 1) == UNSUP


def test_refusals_of_single_operators():
    assert linear(layout=2) == BAD and linear(bt="f16") == BAD and linear(A2=None) == BAD and linear(B2=None) == BAD
    assert linear(A=None) == BAD and linear(B=None) == BAD and linear(bias=P + 2) == ALIGN and linear(bt="bf16", bias=P + 1) == ALIGN
    assert linear(layout="RR", ldb=63) == BAD
    assert gated(bt="bf16") == BAD and gated(G=None) == BAD and gated(U=None) == BAD
    assert gated(BG=P + 1) == ALIGN and gated(bt="f32", BU=P + 2) == ALIGN
    assert backward(U=None) == BAD and backward(DU=None) == BAD
    assert weight(acc=2) == BAD and weight(DB=P + 2) == ALIGN and weight(K=0) == UNSUP
    for fn, none in ((linear, "C"), (gated, "Hh"), (backward, "DG")):
        assert fn(K=0, **{none: None}) == BAD                                   # zeros have to go somewhere
        for zero in ("M", "N"):
            assert fn(**{zero: 0, none: None}) == OK
    assert weight(N=0, DW=None) == OK and weight(K=0, DB=None, DW=None) == OK and weight(M=0, DW=None) == BAD
    assert binding.gemm_weight_gradient(None, 1, 1, 1, "bf16", 0, "auto", P, 1, P, 1, P, 1, None, stream=0, check=False) == BAD


# ---- the torch functions' refusals (CPU tensors: nothing is enqueued) --------

def test_binding_refuses_what_is_no_device_matrix():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    for fn in (lambda t: binding.linear(t, t), lambda t: binding.gated(t, t, t), lambda t: binding.gated_backward(t, t, t),
               lambda t: binding.weight_gradient(t, t)):
        for bad in (x, x.float(), x[0], x.to(torch.int8), None, [1]):
            with pytest.raises(ValueError):
                fn(bad)


def test_binding_refuses_names():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    for kw in (dict(layout="CR"), dict(activation="tanh"), dict(activation=None), dict(tile="32x32"), dict(pair=x), dict(pair=(x,)),
               dict(pair=(x, None))):
        with pytest.raises(ValueError):
            binding.linear(x, x, **kw)
    for fn in (lambda **kw: binding.gated(x, x, x, **kw), lambda **kw: binding.gated_backward(x, x, x, **kw)):
        for kw in (dict(activation="swish"), dict(tile="512x512")):
            with pytest.raises(ValueError):
                fn(**kw)
