"""The feed-forward operators on the GPU against their definitions in 64 bits:
every tile class, type and load path at ragged sizes, every activation on every
16-bit value, rows at any address, empty sizes."""
import pytest
import torch

from software_pipelined_tiled_02_amd import binding
from tests import linear_ref as R
from tests.linear_ref import FT, assert_within, place

pytestmark = pytest.mark.gpu

TILES = ("256x256", "128x256", "128x128", "64x64", "64x64k4", "64x32", "32x32", "16x32", "16x16")


def rand(g, rows, cols, dtype, size=1.0):
    return (size * torch.randn((rows, cols), generator=g, device="cuda")).to(FT[dtype])


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows16(t):
    """t in rows that start on 16 bytes, NaNs between them."""
    return place(t, (t.shape[1] + 7) // 8 * 8)


def check_linear(a, b, c, z, dtype, layout="RC", bias=None, activation="none", residual=None, pair=None, what=""):
    turn = (lambda t: t.double().t()) if layout == "RC" else (lambda t: t.double())
    ref, off, zref, zoff = R.linear(a.double(), turn(b), dtype, None if bias is None else bias.double(), activation,
                                    None if residual is None else residual.double(),
                                    None if pair is None else (pair[0].double(), turn(pair[1])))
    assert_within(c, ref, off, "c " + what)
    if z is not None:
        assert_within(z, zref, zoff, "z " + what)


# ---- linear -----------------------------------------------------------------

@pytest.mark.parametrize("dtype", ("bf16", "f16"))
@pytest.mark.parametrize("layout", ("RC", "RR"))
@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("M,N,K", ((1, 1, 1), (300, 264, 200), (257, 520, 64), (70, 130, 129), (33, 65, 63), (512, 40, 330)))
def test_linear_every_class(M, N, K, tile, layout, dtype):
    g = gen(1)
    a, b = rand(g, M, K, dtype), rand(g, *((N, K) if layout == "RC" else (K, N)), dtype, K ** -0.5)
    r, bias = rand(g, M, N, dtype), torch.randn(N, generator=g, device="cuda")
    c, z = binding.linear(rows16(a), rows16(b), layout=layout, bias=bias, activation="gelu", residual=r, keep=True, tile=tile)
    check_linear(a, b, c, z, dtype, layout, bias, "gelu", r, what=tile)


@pytest.mark.parametrize("layout", ("RC", "RR"))
@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("M,N,K,lda,ldb,offset", ((130, 260, 77, 77, None, 0), (70, 67, 130, 131, None, 1), (150, 300, 200, 203, None, 3),
                                                  (65, 7, 5, 5, None, 0), (3, 129, 64, 71, None, 5), (1, 9, 300, 300, None, 1)))
def test_linear_rows_at_any_address(M, N, K, lda, ldb, offset, tile, layout):
    g = gen(2)
    shape = (N, K) if layout == "RC" else (K, N)
    a, b = rand(g, M, K, "bf16"), rand(g, *shape, "bf16", K ** -0.5)
    c = binding.linear(place(a, lda, offset), place(b, shape[1] + offset, 1), layout=layout, tile=tile)
    check_linear(a, b, c, None, "bf16", layout, what=tile)


def on4(t, distance, offset):
    """t in rows on 4 bytes, and not all on 16."""
    assert distance % 2 == 0 and offset % 2 == 0 and (distance % 8 or offset % 8)
    return place(t, distance, offset)


# K: not a multiple of 8 of several K-tiles, exactly one and two of them, less than one, less than 8
@pytest.mark.parametrize("dtype", ("bf16", "f16"))
@pytest.mark.parametrize("layout", ("RC", "RR"))
@pytest.mark.parametrize("tile", TILES + ("auto",))
@pytest.mark.parametrize("M,N,K,lda,ldb,offset", ((300, 262, 202, 202, 6, 0), (70, 100, 64, 66, 0, 2), (257, 130, 128, 128, 10, 4),
                                                  (33, 65, 62, 62, 5, 6), (1, 9, 5, 6, 1, 0), (520, 37, 1004, 1004, 1, 2)))
def test_linear_rows_on_4_bytes(M, N, K, lda, ldb, offset, tile, layout, dtype):
    g = gen(20)
    shape = (N, K) if layout == "RC" else (K, N)
    a, b, a2, b2 = (rand(g, *s, dtype, z) for s, z in ((( M, K), 1.0), (shape, K ** -0.5)) * 2)
    r, bias = rand(g, M, N, dtype), torch.randn(N, generator=g, device="cuda")
    ldb = (shape[1] + ldb) // 2 * 2
    at = on4(a, lda, offset + 2 * (lda % 8 == 0 and offset % 8 == 0)), place(b, ldb, 2)
    c, z = binding.linear(*at, layout=layout, bias=bias, activation="gelu", residual=r, keep=True, tile=tile)
    check_linear(a, b, c, z, dtype, layout, bias, "gelu", r, what=tile)
    c = binding.linear(*at, layout=layout, pair=(rows16(a2), place(b2, ldb + 4, 4)), tile=tile)
    check_linear(a, b, c, None, dtype, layout, pair=(a2, b2), what=tile)


@pytest.mark.parametrize("tile", TILES + ("auto",))
@pytest.mark.parametrize("M,N,K", ((300, 140, 202), (65, 33, 64), (1, 1, 2), (257, 18, 129), (40, 200, 1004)))
def test_others_of_rows_on_4_bytes(M, N, K, tile):
    g, dtype = gen(21), "bf16"
    even = lambda n: (n + 1) // 2 * 2  # noqa: E731
    x, wg, wu = rand(g, M, K, dtype), rand(g, N, K, dtype, K ** -0.5), rand(g, N, K, dtype, K ** -0.5)
    if tile in TILES[:-1] + ("auto",):
        got = binding.gated(on4(x, even(K) + 2, 2), rows16(wg), place(wu, even(K), 4), keep=True, tile=tile)
        for v, (want, off), name in zip(got, R.gated(x.double(), wg.double(), wu.double(), dtype, "silu"), "hgu"):
            assert_within(v, want, off, name)
    w, gate, up = rand(g, K, N, dtype, K ** -0.5), rand(g, M, N, dtype, 2.0), rand(g, M, N, dtype)
    for at in ((on4(x, even(K), 2), rows16(w)), (rows16(x), on4(w, even(N), 6)), (on4(x, even(K) + 4, 2), on4(w, even(N) + 6, 2))):
        got = binding.gated_backward(*at, gate, up, keep=True, tile=tile)
        for v, (want, off) in zip(got, R.gated_backward(x.double(), w.double(), gate.double(), up.double(), dtype, "silu")):
            assert_within(v, want, off, tile)
    if tile not in TILES[7:]:
        dc = rand(g, M, N, dtype)
        dw, off, db, db_off = R.weight_gradient(dc.double(), x.double())
        for at in ((on4(dc, even(N), 2), rows16(x)), (rows16(dc), on4(x, even(K), 6)), (on4(dc, even(N) + 2, 4), on4(x, even(K) + 4, 2))):
            got, sums = binding.weight_gradient(*at, bias=True, tile=tile)
            assert_within(got, dw, off, "dw")
            assert_within(sums, db, db_off, "db")


def tight(t):
    """t in rows without a gap, at an address on 2 bytes only; its buffer ends with it."""
    return place(t, t.shape[1], 1)


# rows of odd lengths one behind another, which share dwords; one value, and one more than whole K-tiles of them
@pytest.mark.parametrize("dtype", ("bf16", "f16"))
@pytest.mark.parametrize("tile", TILES + ("auto",))
@pytest.mark.parametrize("M,N,K", ((65, 1, 129), (129, 33, 65), (1, 257, 193), (200, 65, 1), (130, 7, 257), (67, 131, 64), (257, 263, 321)))
def test_odd_rows_without_a_gap(M, N, K, tile, dtype):
    g = gen(22)
    x, w, w2 = rand(g, M, K, dtype), rand(g, N, K, dtype, K ** -0.5), rand(g, N, K, dtype, K ** -0.5)
    r, up = rand(g, M, N, dtype), rand(g, M, N, dtype)
    rr, rr2 = w.t().contiguous(), w2.t().contiguous()
    check_linear(x, w, binding.linear(tight(x), tight(w), residual=tight(r), tile=tile), None, dtype, residual=r, what="RC")
    check_linear(x, rr, binding.linear(tight(x), tight(rr), layout="RR", tile=tile), None, dtype, "RR", what="RR")
    check_linear(x, rr, binding.linear(tight(x), tight(rr), layout="RR", pair=(tight(x), tight(rr2)), tile=tile), None, dtype, "RR",
                 pair=(x, rr2), what="pair")
    if tile != "16x16":
        for v, (want, off), name in zip(binding.gated(tight(x), tight(w), tight(w2), keep=True, tile=tile),
                                        R.gated(x.double(), w.double(), w2.double(), dtype, "silu"), "hgu"):
            assert_within(v, want, off, name)
    for v, (want, off) in zip(binding.gated_backward(tight(x), tight(rr), tight(r), tight(up), keep=True, tile=tile),
                              R.gated_backward(x.double(), rr.double(), r.double(), up.double(), dtype, "silu")):
        assert_within(v, want, off, "backward")
    if tile not in TILES[7:]:
        # K tokens of an N x M weight
        dw, off, db, db_off = R.weight_gradient(rr.double(), x.double().t())
        got, sums = binding.weight_gradient(tight(rr), tight(x.t().contiguous()), bias=True, tile=tile)
        assert_within(got, dw, off, "dw")
        assert_within(sums, db, db_off, "db")


@pytest.mark.parametrize("layout", ("RC", "RR"))
@pytest.mark.parametrize("tile", TILES + ("auto",))
@pytest.mark.parametrize("M,N,K,odd", ((300, 280, 136, False), (65, 72, 67, False), (129, 100, 203, True), (20, 33, 64, True), (40, 40, 7, True)))
def test_linear_two_products(M, N, K, odd, tile, layout):
    g, shape = gen(3), (N, K) if layout == "RC" else (K, N)
    ms = [rand(g, M, K, "bf16"), rand(g, *shape, "bf16", K ** -0.5), rand(g, M, K, "bf16"), rand(g, *shape, "bf16", K ** -0.5)]
    r = rand(g, M, N, "bf16")
    # other distances for each
    at = [place(t, (t.shape[1] + 7) // 8 * 8 + (8 * i if not odd else i)) for i, t in enumerate(ms)]
    c = binding.linear(at[0], at[1], layout=layout, pair=(at[2], at[3]), residual=r, tile=tile)
    check_linear(ms[0], ms[1], c, None, "bf16", layout, residual=r, pair=(ms[2], ms[3]), what=tile)


@pytest.mark.parametrize("activation", R.ACTIVATIONS)
@pytest.mark.parametrize("dtype", ("bf16", "f16"))
def test_activation_of_every_value(dtype, activation):
    """A sum of one product with 1: every 16-bit pattern goes through, infinities and NaNs among them."""
    x = torch.arange(-32768, 32768, dtype=torch.int16, device="cuda").view(FT[dtype])[:, None]
    one = torch.ones((1, 1), dtype=FT[dtype], device="cuda")
    c, z = binding.linear(x, one, activation=activation, keep=True)
    ref = R.act(x.double(), activation)
    keep = ref.abs() <= torch.finfo(FT[dtype]).max
    tiny = 2.0 ** -126                                     # fp32's subnormals may be flushed
    off = R.ACT * ref.abs() + tiny + R.flushed(x.double())
    assert_within(c[keep], ref[keep], (off + R.half_step(ref.abs() + off, dtype))[keep], activation)
    rest = ~keep
    assert torch.equal(c[rest].isnan(), ref[rest].isnan()) and bool((c[rest].double() == ref[rest])[~ref[rest].isnan()].all())
    finite = x.isfinite()
    assert bool(((z.double() - x.double()).abs() <= tiny)[finite].all()) and torch.equal(z.isnan(), x.isnan())


@pytest.mark.parametrize("activation", R.ACTIVATIONS)
@pytest.mark.parametrize("dtype", ("bf16", "f16"))
def test_derivative_at_every_value(dtype, activation):
    x = torch.arange(-32768, 32768, dtype=torch.int16, device="cuda").view(FT[dtype])[:, None]
    one = torch.ones((65536, 1), dtype=FT[dtype], device="cuda")
    dz, h = binding.gated_backward(one, one[:1], x, activation=activation, keep=True)
    ref, terms = R.slope(x.double(), activation)
    finite = x.isfinite()[:, 0]
    off = R.ACT * terms + R.flushed(x.double(), of_slope=True)
    assert_within(dz[finite], ref[finite], (off + R.half_step(ref.abs() + off, dtype))[finite], activation)
    nans = x.isnan()
    assert bool((dz[nans] == 1).all() if activation == "none" else dz[nans].isnan().all())    # (a constant, or a NaN)
    a = R.act(x.double(), activation)[finite]
    off = R.ACT * a.abs() + R.flushed(x.double())[finite]
    assert_within(h[finite], a, off + R.half_step(a.abs() + off, dtype), activation)


def test_linear_in_place_of_its_residual():
    g = gen(4)
    a, b, r = rand(g, 200, 136, "f16"), rand(g, 203, 136, "f16", 0.1), rand(g, 200, 203, "f16")
    want = binding.linear(a, b, residual=r, activation="silu")
    got = binding.linear(a, b, residual=r, activation="silu", out=r)
    assert got is r and torch.equal(got, want)


@pytest.mark.parametrize("tile", TILES)
def test_a_nan_stays_in_its_row_and_column(tile):
    g = gen(5)
    a, b = rand(g, 150, 200, "bf16"), rand(g, 170, 200, "bf16")
    want = binding.linear(a, b, tile=tile)
    a[17, 199], b[33, 3] = float("nan"), float("inf")
    got = binding.linear(a, b, tile=tile)
    assert bool(got[17].isnan().all()) and not bool(got[:, 33].isfinite().any())
    rows, cols = torch.arange(150, device="cuda") != 17, torch.arange(170, device="cuda") != 33
    assert torch.equal(got[rows][:, cols], want[rows][:, cols])


def test_outputs_and_what_lies_around_them():
    """Padded outputs: what lies between and behind the rows is left as it was."""
    g = gen(6)
    M, N, K = 70, 101, 96
    a, b = rand(g, M, K, "bf16"), rand(g, N, K, "bf16")
    for ld, off in ((N, 0), (N + 3, 1), (N + 27, 5)):
        buf = torch.full((off + M * ld + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[off:].as_strided((M, N), (ld, 1))
        c = binding.linear(a, b, out=out)
        assert c is out and torch.equal(c, binding.linear(a, b))
        mask = torch.ones_like(buf, dtype=torch.bool)
        mask[off:].as_strided((M, N), (ld, 1)).fill_(False)
        assert bool((buf[mask] == 7.0).all())


def test_empty_sizes():
    d, t = "cuda", torch.bfloat16
    e = lambda *s: torch.ones(s, dtype=t, device=d)  # noqa: E731
    bias, r = torch.full((9,), -2.0, device=d), e(5, 9)
    c, z = binding.linear(e(5, 0), e(9, 0), bias=bias, activation="relu", residual=r, keep=True)
    assert bool((c == 1).all()) and bool((z == -2).all())
    c = binding.linear(e(5, 0), e(0, 9), layout="RR", pair=(e(5, 0), e(0, 9)))
    assert bool((c == 0).all())
    assert binding.linear(e(0, 8), e(9, 8), pair=(e(0, 8), e(9, 8))).shape == (0, 9)
    assert binding.linear(e(5, 8), e(0, 8)).shape == (5, 0)
    h, g, u = binding.gated(e(3, 0), e(9, 0), e(9, 0), gate_bias=bias, keep=True)
    assert bool((g == -2).all()) and bool((u == 0).all()) and bool((h == 0).all())
    assert binding.gated(e(0, 4), e(9, 4), e(9, 4)).shape == (0, 9)
    dg, du, h = binding.gated_backward(e(4, 0), e(0, 9), e(4, 9), e(4, 9), keep=True)
    assert bool((dg == 0).all()) and bool((du == 0).all()) and bool((h > 0.7).all())
    assert binding.gated_backward(e(0, 3), e(3, 9), e(0, 9)).shape == (0, 9)
    dw, db = binding.weight_gradient(e(0, 9), e(0, 20), bias=True)
    assert dw.shape == (9, 20) and bool((dw == 0).all()) and bool((db == 0).all())
    out, s = torch.full((9, 20), 3.0, device=d), torch.full((9,), 4.0, device=d)
    binding.weight_gradient(e(0, 9), e(0, 20), out=out, bias_out=s, accumulate=True)
    assert bool((out == 3).all()) and bool((s == 4).all())
    assert binding.weight_gradient(e(4, 0), e(4, 5)).shape == (0, 5)
    assert binding.weight_gradient(e(4, 5), e(4, 0)).shape == (5, 0)


# ---- gated ------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ("bf16", "f16"))
@pytest.mark.parametrize("tile", TILES[:-1] + ("auto",))
@pytest.mark.parametrize("M,N,K,odd", ((300, 140, 200, False), (65, 33, 64, False), (1, 1, 1, False), (257, 17, 129, False),
                                       (130, 200, 77, True), (31, 64, 128, True), (1, 3, 9, True)))
def test_gated(M, N, K, odd, tile, dtype):
    g = gen(7)
    x, wg, wu = rand(g, M, K, dtype), rand(g, N, K, dtype, K ** -0.5), rand(g, N, K, dtype, K ** -0.5)
    bg, bu = (torch.randn(N, generator=g, device="cuda").to(FT[dtype]) for _ in range(2))
    at = [place(t, K + 3, i) for i, t in enumerate((x, wg, wu))] if odd else [rows16(t) for t in (x, wg, wu)]
    got = binding.gated(*at, gate_bias=bg, up_bias=bu, keep=True, tile=tile)
    ref = R.gated(x.double(), wg.double(), wu.double(), dtype, "silu", bg.double(), bu.double())
    for v, (want, off), name in zip(got, ref, "hgu"):
        assert_within(v, want, off, name)
    h = binding.gated(*at, activation="gelu_tanh", tile=tile)
    assert_within(h, *R.gated(x.double(), wg.double(), wu.double(), dtype, "gelu_tanh")[0], "h")


# ---- gated_backward ----------------------------------------------------------

@pytest.mark.parametrize("dtype", ("bf16", "f16"))
@pytest.mark.parametrize("gate", (True, False))
@pytest.mark.parametrize("tile", TILES + ("auto",))
@pytest.mark.parametrize("M,N,K,odd", ((300, 264, 200, False), (65, 67, 64, False), (1, 1, 1, False), (130, 201, 77, True),
                                       (31, 6, 128, True), (2, 130, 3, True)))
def test_gated_backward(M, N, K, odd, tile, gate, dtype):
    rng = gen(8)
    dy, w = rand(rng, M, K, dtype, 0.1), rand(rng, K, N, dtype, K ** -0.5)
    g, u = rand(rng, M, N, dtype, 2.0), rand(rng, M, N, dtype) if gate else None
    at = [place(dy, K + 1, 1), place(w, N + 1, 3)] if odd else [rows16(dy), rows16(w)]
    gu = [place(g, N + 5, 1), None if u is None else place(u, N + 2, 3)]
    for activation in ("silu", "gelu") if tile == "auto" else ("silu",):
        got = binding.gated_backward(*at, *gu, activation=activation, keep=True, tile=tile)
        ref = R.gated_backward(dy.double(), w.double(), g.double(), None if u is None else u.double(), dtype, activation)
        assert len(got) == len(ref)
        for v, (want, off) in zip(got, ref):
            assert_within(v, want, off, activation)
        without = binding.gated_backward(*at, *gu, activation=activation, tile=tile)
        without = without if gate else (without,)
        assert len(without) == len(got) - 1 and all(torch.equal(a, b) for a, b in zip(without, got))


# ---- weight_gradient ----------------------------------------------------------

@pytest.mark.parametrize("dtype", ("bf16", "f16"))
@pytest.mark.parametrize("tile", TILES[:7] + ("auto",))
@pytest.mark.parametrize("M,N,K,odd", ((200, 300, 264, False), (64, 257, 130, False), (1, 70, 33, False), (129, 1, 1, False),
                                       (330, 129, 513, False), (77, 130, 201, True), (65, 9, 6, True), (1, 31, 67, True), (3, 2, 130, True)))
def test_weight_gradient(M, N, K, odd, tile, dtype):
    g = gen(9)
    dc, a = rand(g, M, N, dtype), rand(g, M, K, dtype)
    at = [place(dc, N + 1, 1), place(a, K + 3, 3)] if odd else [rows16(dc), rows16(a)]
    dw, off, db, db_off = R.weight_gradient(dc.double(), a.double())
    got, sums = binding.weight_gradient(*at, bias=True, tile=tile)
    assert_within(got, dw, off, "dw")
    assert_within(sums, db, db_off, "db")
    assert torch.equal(binding.weight_gradient(*at, tile=tile), got)
    base = torch.randn((N, K + 2), generator=g, device="cuda")
    out, more = base.clone()[:, :K], torch.ones(N, device="cuda")
    r = binding.weight_gradient(*at, out=out, bias_out=more, accumulate=True, tile=tile)
    assert r[0] is out and r[1] is more
    want = dw + base[:, :K].double()
    assert_within(out, want, off + 2 * R.U * want.abs(), "dw added")
    assert_within(more, db + 1, db_off + 2 * R.U * (db + 1).abs(), "db added")
