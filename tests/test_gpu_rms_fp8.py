"""gemm_rms_fp8 and gemm_rms_backward on the GPU against their definitions in 64 bits.

Bounds.  h is one fp32 addition and one rounding, which torch does alike: equal
bits.  rstd: a sum of D squares, each term's error and the chain below
(D / 8 + 16) u in the kernel's order (a thread's values in turn, then the lanes), a
division, a sum, a root and a division: within (D / 8 + 20) u relative, half of
it after the root; held to (D / 8 + 20) u.  y: three roundings more.  A value in 8 bits is off by
half a step of its block's scale (2^-4 of the value, e5m2 2^-3; below the
smallest normal half a step of it) beyond y's own error.
"""
import numpy as np
import pytest
import torch

from software_pipelined_tiled_02_amd import binding
from tests import fp8_ref as R
from tests.fp8_util import FT, raw_of

pytestmark = pytest.mark.gpu

SIZES = ((1, 1), (1, 8), (5, 100), (3, 512), (9, 520), (2, 1024), (4, 1025), (3, 2048), (2, 2056), (5, 4096), (2, 4104),
         (1, 8192), (2, 8200), (1, 16384), (2, 16392), (1, 32768), (300, 128))
STEP = {"e4m3": (2.0 ** -4, 2.0 ** -10), "e5m2": (2.0 ** -3, 2.0 ** -17)}     # half steps: relative, of subnormals


def inputs(M, D, x, w, residual, seed=0):
    g = torch.Generator().manual_seed(seed + 31 * M + D)
    t = torch.randn((M, D), generator=g).to(FT[x])
    r = (2 * torch.randn((M, D), generator=g)).to(FT[x]) if residual else None
    return t, r, (1 + 0.3 * torch.randn((D,), generator=g)).to(FT[w])


def check_forward(t, r, wt, out, fp8, pow2, eps, x):
    q, s, h, rstd = (o.cpu() for o in out[:4])
    M, D = t.shape
    href = t if r is None else (t.float() + r.float()).to(t.dtype)
    assert torch.equal(h.view(torch.uint8), href.contiguous().view(torch.uint8))
    y, rs = R.rms(href.double().numpy(), None, wt.double().numpy(), eps)
    rel = (D / 8 + 20) * R.U
    R.assert_within(rstd.double().numpy(), rs, rs * rel, "rstd")
    rel_y = rel + 4 * R.U
    s_ref = np.maximum(R.block_amax(y, 1) / R.TOP[fp8], 2.0 ** -126)
    sv = s.double().numpy()
    if pow2:
        assert np.array_equal(np.frexp(sv)[0], np.full_like(sv, 0.5))
        assert (sv >= s_ref * (1 - rel_y - 2 * R.U)).all() and (sv < 2 * s_ref * (1 + rel_y + 2 * R.U)).all()
    else:
        R.assert_within(sv, s_ref, s_ref * (rel_y + 2 * R.U), "scales")
    at = R.spread(sv, 1, M, D)
    bound = np.maximum(np.abs(y) * STEP[fp8][0], at * STEP[fp8][1]) * (1 + 2.0 ** -10) + np.abs(y) * (rel_y + 4 * R.U)
    R.assert_within(R.decode(raw_of(q), fp8) * at, y, bound, "q")
    if len(out) > 4:
        R.assert_within(out[4].cpu().double().numpy(), y, R.half_step(y, x) * (1 + 2.0 ** -8) + np.abs(y) * rel_y, "y")


@pytest.mark.parametrize("M,D", SIZES)
def test_forward_sizes(M, D):
    for residual in (False, True):
        t, r, w = inputs(M, D, "bf16", "bf16", residual)
        out = binding.rms_fp8(t.cuda(), w.cuda(), residual=None if r is None else r.cuda(), norm=True)
        check_forward(t, r, w, out, "e4m3", False, 1e-6, "bf16")


@pytest.mark.parametrize("x,w", (("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")))
@pytest.mark.parametrize("fp8,pow2", (("e4m3", False), ("e5m2", True)))
def test_forward_types(x, w, fp8, pow2):
    for M, D in ((7, 136), (3, 1000), (5, 2500)):
        t, r, wt = inputs(M, D, x, w, True)
        out = binding.rms_fp8(t.cuda(), wt.cuda(), residual=r.cuda(), eps=1e-3, fp8=fp8, pow2=pow2, norm=True)
        check_forward(t, r, wt, out, fp8, pow2, 1e-3, x)


def test_forward_in_place_and_strided():
    M, D = 6, 1032
    t, r, w = inputs(M, D, "bf16", "bf16", True)
    ref = binding.rms_fp8(t.cuda(), w.cuda(), residual=r.cuda())
    for into in ("residual", "x"):
        x, res = t.cuda(), r.cuda()
        out = binding.rms_fp8(x, w.cuda(), residual=res, h_out=res if into == "residual" else x)
        assert out[2].data_ptr() == (res if into == "residual" else x).data_ptr()
        for a, b in zip(out, ref):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    for pad in (3, 8):                                             # rows apart, on and off 16 bytes
        wide = torch.full((M, D + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
        wr, wh = wide.clone(), wide.clone()
        wide[:, :D], wr[:, :D] = t.cuda(), r.cuda()
        out = binding.rms_fp8(wide[:, :D], w.cuda(), residual=wr[:, :D], h_out=wh[:, :D])
        for a, b in zip(out, ref):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
        assert bool(wh[:, D:].isnan().all())
    odd = torch.empty((D + 1,), dtype=torch.bfloat16, device="cuda")[1:]      # a weight off 16 bytes
    odd.copy_(w)
    out = binding.rms_fp8(t.cuda(), odd, residual=r.cuda())
    for a, b in zip(out, ref):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_forward_zeros_and_what_is_not_finite():
    D = 384
    x = torch.zeros((6, D))
    x[1] = 1.0
    x[2, 5] = float("inf")
    x[3, 200] = float("nan")
    x[4, 0] = 1e30                                                 # its square overflows fp32: rstd = 0
    x[5] = 1e-30                                                   # squares vanish beside eps
    w = torch.ones(D)
    q, s, h, rstd = binding.rms_fp8(x.cuda(), w.cuda(), eps=1e-6)
    v = R.decode(raw_of(q), "e4m3") * np.repeat(s.cpu().double().numpy(), 128, 1)
    assert (v[0] == 0).all() and float(rstd[0]) == pytest.approx(1000.0, rel=1e-6)
    assert np.abs(v[1] - 1).max() < 1e-3 and np.isnan(v[2, 5]) and np.isnan(v[3, 200])
    assert float(rstd[2]) == 0 and bool(rstd[3].isnan()) and float(rstd[4]) == 0
    assert np.abs(v[5] / 1e-27 - 1).max() < 0.07
    z = binding.rms_fp8(torch.zeros((2, D), device="cuda"), w.cuda(), eps=0.0)     # 0 * (1 / 0): NaN, as the formula
    assert bool(z[3].isinf().all()) and np.isnan(R.decode(raw_of(z[0]), "e4m3")).all()


def test_forward_rows_without_values():
    """The mean of no values is NaN, as torch has it, whatever the memory held."""
    junk = torch.full((1 << 16,), 3.0, device="cuda")
    del junk
    x, w = torch.empty((5, 0), device="cuda"), torch.empty(0, device="cuda")
    q, s, h, rstd, y = binding.rms_fp8(x, w, norm=True)
    assert q.shape == y.shape == (5, 0) and s.shape == (5, 0) and rstd.shape == (5,) and bool(rstd.isnan().all())
    dx, dw = binding.rms_backward(x, h, w, rstd)
    assert dx.shape == (5, 0) and dw.shape == (0,)
    q, s, h, rstd = binding.rms_fp8(torch.empty((0, 64), device="cuda"), torch.ones(64, device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0, 1) and rstd.shape == (0,)


def check_backward(dy, h, w, rstd, dh, dx, dw, x):
    d = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    M, D = h.shape
    ref, rw = R.rms_backward(d(dy), d(h), d(w), d(rstd), d(dh))
    g, hh, r = np.abs(d(dy) * d(w)), np.abs(d(h)), d(rstd)[:, None]
    # the mean's chain of D terms, its product, and the sums; then one rounding
    err = r * (g * 4 + hh * r * r * (g * hh).mean(1, keepdims=True) * (D / 8 + 24)) * R.U + np.abs(ref) * 2 * R.U
    if dh is not None:
        err = err + np.abs(d(dh)) * 2 * R.U
    R.assert_within(d(dx), ref, err + R.half_step(np.abs(ref) + err, x), "dx")
    err = (np.abs(d(dy)) * hh * r).sum(0) * (M + 20) * R.U
    R.assert_within(d(dw), rw, err + 2.0 ** -126, "dw")


@pytest.mark.parametrize("M,D", SIZES + ((0, 64), (2100, 72), (1500, 1032), (600, 2560), (512, 136), (513, 136), (1100, 4104), (4100, 520), (4096, 200),
                                         (1030, 9000), (1030, 12296), (1030, 12300), (513, 16392), (1025, 7)))
def test_backward_sizes(M, D):
    t, _, w = inputs(M, D, "bf16", "f32", False)
    dy, dh, _ = inputs(M, D, "bf16", "f32", True, seed=5)
    rstd = torch.rsqrt(t.double().square().mean(1) + 1e-6).float()
    for extra in (None, dh):
        dx, dw = binding.rms_backward(dy.cuda(), t.cuda(), w.cuda(), rstd.cuda(), dh=None if extra is None else extra.cuda())
        check_backward(dy, t, w, rstd, extra, dx, dw, "bf16")
        again = binding.rms_backward(dy.cuda(), t.cuda(), w.cuda(), rstd.cuda(), dh=None if extra is None else extra.cuda())
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)      # a fixed order


@pytest.mark.parametrize("x,w", (("bf16", "bf16"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")))
@pytest.mark.parametrize("M,D", ((40, 1100), (1030, 300), (1030, 2052)))
def test_backward_types_strides_and_in_place(M, D, x, w):
    t, _, wt = inputs(M, D, x, w, False)
    dy, dh, _ = inputs(M, D, x, w, True, seed=5)
    rstd = torch.rsqrt(t.double().square().mean(1) + 1e-6).float()
    dx, dw = binding.rms_backward(dy.cuda(), t.cuda(), wt.cuda(), rstd.cuda(), dh=dh.cuda())
    check_backward(dy, t, wt, rstd, dh, dx, dw, x)
    for into in range(3):
        args = [dy.cuda(), t.cuda(), dh.cuda()]
        got, gw = binding.rms_backward(args[0], args[1], wt.cuda(), rstd.cuda(), dh=args[2], dx_out=args[into])
        assert got.data_ptr() == args[into].data_ptr() and torch.equal(got, dx) and torch.equal(gw, dw)
    wide = torch.full((4, M, D + 5), float("nan"), dtype=FT[x], device="cuda")
    for i, v in enumerate((dy, t, dh)):
        wide[i, :, :D] = v.cuda()
    got, gw = binding.rms_backward(wide[0, :, :D], wide[1, :, :D], wt.cuda(), rstd.cuda(), dh=wide[2, :, :D],
                                   dx_out=wide[3, :, :D])
    assert torch.equal(got, dx) and torch.equal(gw, dw) and bool(wide[3, :, D:].isnan().all())


@pytest.mark.parametrize("x", ("f32", "bf16", "f16"))
@pytest.mark.parametrize("M,D", ((1030, 8196), (1030, 8193), (1030, 9300), (1030, 8200), (2000, 10001), (1030, 12284),
                                 (1025, 12287), (1025, 12288), (1025, 12292)))
def test_backward_long_rows_of_every_type(M, D, x):
    """Rows of 8193 and more in groups, which end inside a thread's 8 values and at them:
    contiguous, strided with NaNs between the rows, and in place."""
    t, _, wt = inputs(M, D, x, "f32", False)
    dy, dh, _ = inputs(M, D, x, "f32", True, seed=5)
    rstd = torch.rsqrt(t.double().square().mean(1) + 1e-6).float()
    wt, rs = wt.cuda(), rstd.cuda()
    flat = torch.full(((M + 1) * D,), 7.0, dtype=FT[x], device="cuda")       # what lies behind the last row stays
    dx, dw = binding.rms_backward(dy.cuda(), t.cuda(), wt, rs, dh=dh.cuda(), dx_out=flat[:M * D].view(M, D))
    check_backward(dy, t, wt, rstd, dh, dx, dw, x)
    assert bool((flat[M * D:] == 7.0).all())
    wide = torch.full((4, M, D + 5), float("nan"), dtype=FT[x], device="cuda")
    for i, v in enumerate((dy, t, dh)):
        wide[i, :, :D] = v.cuda()
    got, gw = binding.rms_backward(wide[0, :, :D], wide[1, :, :D], wt, rs, dh=wide[2, :, :D], dx_out=wide[3, :, :D])
    assert torch.equal(got, dx) and torch.equal(gw, dw) and bool(wide[3, :, D:].isnan().all())
    for into in range(3):
        got, gw = binding.rms_backward(wide[0, :, :D], wide[1, :, :D], wt, rs, dh=wide[2, :, :D], dx_out=wide[into, :, :D])
        assert torch.equal(got, dx) and torch.equal(gw, dw) and bool(wide[:, :, D:].isnan().all())
        wide[into, :, :D] = (dy, t, dh)[into].cuda()


def test_backward_is_the_forwards_difference():
    """dx and dw against differences of the forward pass itself, in fp32."""
    M, D, eps = 2, 64, 1e-2
    g = torch.Generator().manual_seed(3)
    x, w, dy = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((M, D), (D,), (M, D)))

    def loss(x, w):
        y = binding.rms_fp8(x.float().cuda(), w.float().cuda(), eps=eps, norm=True)[4]
        return float((y.double().cpu() * dy).sum())

    rstd = binding.rms_fp8(x.float().cuda(), w.float().cuda(), eps=eps)[3]
    dx, dw = binding.rms_backward(dy.float().cuda(), x.float().cuda(), w.float().cuda(), rstd)
    # y is fp32: the loss is off by about 1e-6, which a step of 2^-6 divides by
    # 2^-5; the second-order term is below step^2 * |third derivative| ~ 1e-3
    step = 2.0 ** -6
    for i, j in ((0, 0), (0, 33), (1, 63)):
        d = torch.zeros_like(x)
        d[i, j] = step
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * step) - float(dx[i, j])) < 4e-3
    for j in (1, 40):
        d = torch.zeros_like(w)
        d[j] = step
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * step) - float(dw[j])) < 1e-3


def test_offsets_past_32_bits():
    """Rows 2^30 and more elements apart: row 2 lies past 2^31 elements."""
    M, D, ld = 3, 520, 2 ** 30 + 24
    buf = torch.empty(2 * ld + 8 * D, dtype=torch.bfloat16, device="cuda")
    x, r, w = inputs(M, D, "bf16", "bf16", True)
    dy, dh, _ = inputs(M, D, "bf16", "bf16", True, seed=5)

    def far(i, values=None):
        v = buf.as_strided((M, D), (ld, 1), i * D)
        return v if values is None else v.copy_(values.cuda())

    want = binding.rms_fp8(x.cuda(), w.cuda(), residual=r.cuda(), norm=True)
    got = binding.rms_fp8(far(0, x), w.cuda(), residual=far(1, r), norm=True, h_out=far(2))
    for a, b in zip(got, want):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    dx, dw = binding.rms_backward(dy.cuda(), want[2], w.cuda(), want[3], dh=dh.cuda())
    for into in (far(5), far(3, dy)):                              # beside the others, and in place
        gx, gw = binding.rms_backward(far(3, dy), got[2], w.cuda(), got[3], dh=far(4, dh), dx_out=into)
        assert torch.equal(gx, dx) and torch.equal(gw, dw)


@pytest.mark.parametrize("M,D", ((600, 1032), (1100, 1032)))
def test_backward_captured_and_replayed(M, D):
    """Two graphs of one pool, whose parts of dw share memory, replayed in turn between eager calls."""
    t, _, w = inputs(M, D, "bf16", "bf16", False)
    assert binding.gemm_rms_backward_workspace(M, D) > 0
    dy, dh, _ = (v.cuda() if v is not None else v for v in inputs(M, D, "bf16", "bf16", True, seed=5))
    h, w = t.cuda(), w.cuda()
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    binding.rms_backward(dy, h, w, rstd, dh=dh)                    # eager once: the library
    torch.cuda.synchronize()
    graphs, pool = [], None
    for extra in (dh, None):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            out = binding.rms_backward(dy, h, w, rstd, dh=extra)
        pool = g.pool()
        graphs.append((g, extra, out))
    for i in range(4):
        h.copy_(torch.roll(t, i, 0))
        dy.mul_(-1.25)
        for g, extra, out in graphs:
            want = binding.rms_backward(dy, h, w, rstd, dh=extra)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_two_streams_at_once():
    """Calls that overlap share nothing: each has its own workspace."""
    M, D = 1500, 2048
    sets = []
    for seed in (1, 2):
        t, _, w = inputs(M, D, "bf16", "bf16", False, seed)
        dy, _, _ = inputs(M, D, "bf16", "bf16", False, seed + 10)
        rstd = torch.rsqrt(t.double().square().mean(1) + 1e-6).float()
        args = [v.cuda() for v in (dy, t, w, rstd)]
        sets.append((args, binding.rms_backward(*args)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(6):
        for i in (0, 1):
            got[i].append(binding.rms_backward(*sets[i][0], stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for dx, dw in got[i]:
            assert torch.equal(dx, sets[i][1][0]) and torch.equal(dw, sets[i][1][1])


def test_refusals():
    x = torch.zeros((4, 256), device="cuda")
    w, r = torch.ones(256, device="cuda"), torch.ones(4, device="cuda")
    for call in (lambda: binding.rms_fp8(x.t(), w), lambda: binding.rms_fp8(x, w[:255]),
                 lambda: binding.rms_fp8(x, w.bfloat16()), lambda: binding.rms_fp8(x, w, residual=x[:2]),
                 lambda: binding.rms_fp8(x, w, residual=x.half()), lambda: binding.rms_fp8(x, w, h_out=x.half()),
                 lambda: binding.rms_fp8(x, w, fp8="x"), lambda: binding.rms_fp8(x, w.cpu()),
                 lambda: binding.rms_fp8(x, torch.ones(512, device="cuda")[::2]),
                 lambda: binding.rms_backward(x, x, w, r[:3]), lambda: binding.rms_backward(x.half(), x, w, r),
                 lambda: binding.rms_backward(x, x, w, r, dh=x[:2]), lambda: binding.rms_backward(x, x, w, r.double()),
                 lambda: binding.rms_backward(x, x, w, r, dx_out=x.t())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(binding.GemmError):
        binding.rms_fp8(torch.zeros((1, 32776), device="cuda"), torch.ones(32776, device="cuda"))
    with pytest.raises(binding.GemmError):
        binding.rms_fp8(x, w, eps=-1.0)
