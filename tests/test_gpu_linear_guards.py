"""What lies around the feed-forward operators' results is left as it was: every
output through the C entry points, in rows with gaps, in every class and type, with
256 rows and more behind the last one.  Between the gaps the results are those
of the torch functions, bit for bit; and the same ones again at the next call."""
import pytest
import torch

from software_pipelined_tiled_02_amd import binding
from tests.linear_ref import FT

pytestmark = pytest.mark.gpu
TILES = tuple(binding.LINEAR_TILES)
# whole blocks beside ragged ones, none whole, odd, few rows, one value
SIZES = ((300, 264, 136), (257, 263, 70), (512, 256, 64), (70, 101, 96), (3, 519, 40), (1, 1, 8))
PATTERN = {2: 0x55AA, 4: 0x55AA33CC}


@pytest.fixture(scope="module")
def handle():
    g = binding.Gemm(0)
    yield g.h
    g.close()


def rand(g, rows, cols, dtype, size=1.0):
    return (size * torch.randn((rows, cols), generator=g, device="cuda")).to(FT[dtype])


class Guarded:
    """M x N values, rows N + gap apart, from `lead` values into a buffer of one bit pattern."""

    def __init__(self, M, N, dtype, gap, lead):
        self.M, self.N, self.ld, self.lead = M, N, N + gap, lead
        size = dtype.itemsize
        self.bits = torch.full((lead + (M + 300) * self.ld + 512,), PATTERN[size], dtype={2: torch.int16, 4: torch.int32}[size], device="cuda")
        self.flat = self.bits.view(dtype)
        self.rows = self.flat[lead:].as_strided((M, N), (self.ld, 1))
        self.p = self.flat.data_ptr() + lead * size
        self.size = size

    def check(self, want, what):
        assert torch.equal(self.rows, want), what
        outside = torch.ones_like(self.bits, dtype=torch.bool)
        outside[self.lead:].as_strided((self.M, self.N), (self.ld, 1)).fill_(False)
        assert bool((self.bits[outside] == PATTERN[self.size]).all()), "around " + what


GAPS = ((0, 1), (3, 5), (8, 8), (24, 16))


def outputs(M, N, dtype, names):
    """One buffer for each name, with gaps and leads of several kinds."""
    return {n: Guarded(M, N, FT[dtype], *GAPS[(i + M) % len(GAPS)]) for i, n in enumerate(names)}


@pytest.mark.parametrize("dtype", ("bf16", "f16"))
@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_around_linear(M, N, K, tile, dtype, handle):
    g = torch.Generator(device="cuda").manual_seed(40)
    a, r, bias = rand(g, M, K, dtype), rand(g, M, N, dtype), torch.randn(N, generator=g, device="cuda")
    for layout in ("RC", "RR"):
        b = rand(g, *((N, K) if layout == "RC" else (K, N)), dtype, K ** -0.5)
        c, z = binding.linear(a, b, layout=layout, bias=bias, activation="silu", residual=r, keep=True, tile=tile)
        for _ in range(2):
            o = outputs(M, N, dtype, "cz")
            binding.gemm_linear(handle, M, N, K, dtype, layout, "silu", "f32", tile, a, K, b, b.shape[1], None, 0, None, 0, bias, r, N,
                                o["z"].p, o["z"].ld, o["c"].p, o["c"].ld, torch.cuda.current_stream())
            o["c"].check(c, "c")
            o["z"].check(z, "z")
        o = outputs(M, N, dtype, "c")["c"]                   # over its residual
        o.rows.copy_(r)
        binding.gemm_linear(handle, M, N, K, dtype, layout, "silu", "f32", tile, a, K, b, b.shape[1], None, 0, None, 0, bias, o.p, o.ld,
                            None, 0, o.p, o.ld, torch.cuda.current_stream())
        o.check(c, "c in place")


@pytest.mark.parametrize("dtype", ("bf16", "f16"))
@pytest.mark.parametrize("tile", [t for t in TILES if t != "16x16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_around_gated(M, N, K, tile, dtype, handle):
    g = torch.Generator(device="cuda").manual_seed(41)
    x, wg, wu = rand(g, M, K, dtype), rand(g, N, K, dtype, K ** -0.5), rand(g, N, K, dtype, K ** -0.5)
    want = dict(zip("hgu", binding.gated(x, wg, wu, keep=True, tile=tile)))
    for _ in range(2):
        o = outputs(M, N, dtype, "hgu")
        binding.gemm_gated(handle, M, N, K, dtype, "silu", "f32", tile, x, K, wg, K, wu, K, None, None, o["g"].p, o["g"].ld, o["u"].p,
                           o["u"].ld, o["h"].p, o["h"].ld, torch.cuda.current_stream())
        for name in want:
            o[name].check(want[name], name)


@pytest.mark.parametrize("dtype", ("bf16", "f16"))
@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_around_gated_backward(M, N, K, tile, dtype, handle):
    g = torch.Generator(device="cuda").manual_seed(42)
    dy, w = rand(g, M, K, dtype), rand(g, K, N, dtype, K ** -0.5)
    gate, up = rand(g, M, N, dtype), rand(g, M, N, dtype)
    for u in (up, None):
        names = ("dg", "du", "h") if u is not None else ("dg", "h")
        want = dict(zip(names, binding.gated_backward(dy, w, gate, u, keep=True, tile=tile)))
        o = outputs(M, N, dtype, names)
        du = o.get("du")
        binding.gemm_gated_backward(handle, M, N, K, dtype, "silu", tile, dy, K, w, N, gate, N, u, N, o["dg"].p, o["dg"].ld,
                                    du and du.p, du.ld if du else 0, o["h"].p, o["h"].ld, torch.cuda.current_stream())
        for name in names:
            o[name].check(want[name], name)


@pytest.mark.parametrize("dtype", ("bf16", "f16"))
@pytest.mark.parametrize("tile", TILES[:8])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_around_weight_gradient(M, N, K, tile, dtype, handle):
    """M x N the weight, K tokens; written, then added to."""
    g = torch.Generator(device="cuda").manual_seed(43)
    dc, a = rand(g, K, M, dtype), rand(g, K, N, dtype)
    dw, db = binding.weight_gradient(dc, a, bias=True, tile=tile)
    o, s = Guarded(M, N, torch.float32, 3 + M % 2, 5), Guarded(1, M, torch.float32, 0, 3)
    for add in (0, 1):
        binding.gemm_weight_gradient(handle, K, M, N, dtype, add, tile, dc, M, a, N, o.p, o.ld, s.p, torch.cuda.current_stream())
        o.check(dw * (1 + add), "dw")                        # (doubled without a rounding)
        s.check((db * (1 + add))[None], "db")


def test_every_operator_repeats_its_bits():
    """Few rows too, where waves of one workgroup share K; beside other work on another stream."""
    g = torch.Generator(device="cuda").manual_seed(44)
    side, junk = torch.cuda.Stream(), torch.zeros(2 ** 24, device="cuda")
    for M, N, K in ((1, 4096, 2048), (64, 1024, 2048), (500, 1032, 1028)):
        x, wg, wu = rand(g, M, K, "bf16"), rand(g, N, K, "bf16", K ** -0.5), rand(g, N, K, "bf16", K ** -0.5)
        dy, gate, up = rand(g, M, K, "bf16"), rand(g, M, N, "bf16"), rand(g, M, N, "bf16")
        wd = wg.t().contiguous()

        def every():
            return (binding.linear(x, wg, activation="gelu"), *binding.gated(x, wg, wu, keep=True),
                    *binding.gated_backward(dy, wd, gate, up, keep=True), binding.linear(gate, wg, layout="RR", pair=(up, wu)),
                    *binding.weight_gradient(gate, x, bias=True))

        first = every()
        for _ in range(10):
            with torch.cuda.stream(side):
                junk.add_(1.0)
            assert all(torch.equal(a, b) for a, b in zip(every(), first)), (M, N, K)
