"""The 8-bit operators at the ends of what they take: strides at the border of
the 32-bit offsets, the most rows, every class of the norm in every type, one
tensor in several places, and other streams.  Bounds as in the tests of each operator."""
import subprocess
import sys

import numpy as np
import pytest
import torch

from software_pipelined_tiled_02_amd import binding
from tests import fp8_ref as R
from tests.conftest import ROOT
from tests.fp8_util import F8, FT, check_product, f8_of, operand, raw_of, values
from tests.test_gpu_rms_fp8 import check_backward, check_forward, inputs

pytestmark = pytest.mark.gpu


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---- the product ------------------------------------------------------------

@pytest.mark.parametrize("tile,rows", (("256x256", 1), ("256x128", 128), ("128x128", 1), ("64x64", 1), ("64x32", 128), ("32x32", 1)))
def test_scales_at_the_border_of_their_range(tile, rows):
    """256 rows of scales 2^20 floats apart, the second block 2^27 - 1 on: just below 2^31 bytes."""
    M, N, K = 256, 256, 256
    rng = np.random.default_rng(5)
    a, sa = operand(rng, M, K, "e4m3", 1)
    b, sb = operand(rng, N, K, "e4m3", rows)
    far = []
    for s in (sa, sb):
        t = torch.zeros(255 * 2 ** 20 + 2 ** 27, device="cuda").as_strided(s.shape, (2 ** 20, 2 ** 27 - 1))
        far.append(t.copy_(torch.from_numpy(s).cuda()))
    c = binding.run_fp8(f8_of(a, "e4m3"), far[0], f8_of(b, "e4m3"), far[1], tile=tile)
    check_product(c, a, sa, b, sb, "e4m3", "e4m3", rows, "bf16", tile)


def test_rows_too_far_apart_for_most_tiles():
    """Rows 2^25 bytes apart: the tiles of 64 rows do not reach, those of 32 do."""
    M, N, K, ld = 70, 2500, 1030, 1 << 25
    assert binding.gemm_query_fp8(M, N, K)[1]["block_m"] == 64
    assert binding.gemm_query_fp8(M, N, K, lda=ld)[1]["block_m"] == 32
    rng = np.random.default_rng(6)
    a, sa = operand(rng, M, K, "e4m3", 1)
    b, sb = operand(rng, N, K, "e4m3", 128)
    wide = torch.empty((M - 1) * ld + K, dtype=torch.uint8, device="cuda").as_strided((M, K), (ld, 1))
    wide.copy_(torch.from_numpy(a).cuda())
    flat = f8_of(np.pad(b, ((0, 0), (0, 10))), "e4m3")[:, :K]
    c = binding.run_fp8(wide.view(F8["e4m3"]), torch.from_numpy(sa).cuda(), flat, torch.from_numpy(sb).cuda())
    check_product(c, a, sa, b, sb, "e4m3", "e4m3", 128, "bf16", "far rows")


@pytest.mark.parametrize("swap", (False, True))
def test_millions_of_rows(swap):
    """A tall and a wide product; sampled rows, the last one among them."""
    M, N, K = 2 ** 21 + 3, 5, 40
    g = torch.Generator(device="cuda").manual_seed(3)
    raw = torch.randint(0, 0x78, (M, 48), generator=g, device="cuda", dtype=torch.uint8)       # finite values
    s = torch.rand((M, 1), generator=g, device="cuda") + 0.5
    b, sb = operand(np.random.default_rng(1), N, K, "e4m3", 1)
    at = torch.cat([torch.tensor([0, 1, 2 ** 20, M - 4, M - 2, M - 1]), torch.arange(7, M, 50021)]).cuda()
    a8, b8, tb = raw.view(F8["e4m3"])[:, :K], f8_of(np.pad(b, ((0, 0), (0, 8))), "e4m3")[:, :K], torch.from_numpy(sb).cuda()
    a_s, s_s = raw[at][:, :K].cpu().numpy(), s[at].cpu().numpy()
    if swap:
        c = binding.run_fp8(b8, tb, a8, s)[:, at]
        check_product(c, b, sb, a_s, s_s, "e4m3", "e4m3", 1, "bf16", "wide")
    else:
        c = binding.run_fp8(a8, s, b8, tb)[at]
        check_product(c, a_s, s_s, b, sb, "e4m3", "e4m3", 1, "bf16", "tall")


# ---- quantisation -----------------------------------------------------------

@pytest.mark.parametrize("block", ("row", "tile"))
def test_quantize_millions_of_rows(block):
    M, K, rows = 2 ** 20 + 5, 3, binding.BLOCK_ROWS[block]
    x = values(np.random.default_rng(2), M, K)
    q, s, qt, st = binding.quantize_fp8(torch.from_numpy(x).cuda(), block=block, transpose=True)
    for got, scale, src in ((q, s, x), (qt, st, np.ascontiguousarray(x.T))):
        ref, want = R.quantize_fp32(src, "e4m3", rows)
        assert np.array_equal(raw_of(got), ref) and np.array_equal(scale.cpu().numpy(), want)


# ---- the norm ---------------------------------------------------------------

@pytest.mark.parametrize("x,w", (("bf16", "f32"), ("f16", "f16"), ("f32", "f32")))
@pytest.mark.parametrize("M,D", ((600, 520), (513, 1023), (520, 1025), (513, 2049), (513, 4097), (514, 8191), (513, 8193),
                                 (3, 4097), (3, 8191), (3, 16383), (2, 16385), (2, 32767)))
def test_norm_every_class_in_every_type(M, D, x, w):
    t, r, wt = inputs(M, D, x, w, True)
    out = binding.rms_fp8(t.cuda(), wt.cuda(), residual=r.cuda(), norm=True)
    check_forward(t, r, wt, out, "e4m3", False, 1e-6, x)


@pytest.mark.parametrize("x", ("f16", "f32"))
@pytest.mark.parametrize("M,D", ((3, 4097), (600, 4097), (3, 8191), (1100, 4095), (1100, 8191), (600, 16383), (1100, 16384),
                                 (1100, 16385), (2, 32767), (600, 32767)))
def test_norm_backward_every_class_in_every_type(M, D, x):
    t, _, w = inputs(M, D, x, x, False)
    dy, dh, _ = inputs(M, D, x, x, True, seed=5)
    rstd = torch.rsqrt(t.double().square().mean(1) + 1e-6).float()
    dx, dw = binding.rms_backward(dy.cuda(), t.cuda(), w.cuda(), rstd.cuda(), dh=dh.cuda())
    check_backward(dy, t, w, rstd, dh, dx, dw, x)


def test_norm_of_the_most_rows():
    """GEMM_RMS_MAX_ROWS rows: sampled ones against the definition, dw over all of them."""
    M, D = binding.GEMM_RMS_MAX_ROWS, 24
    g = torch.Generator(device="cuda").manual_seed(4)
    x, r, dy = (torch.randn((M, D), generator=g, device="cuda").bfloat16() for _ in range(3))
    w = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).bfloat16()
    out = binding.rms_fp8(x, w, residual=r, norm=True)
    at = torch.cat([torch.tensor([0, 1, M - 2, M - 1]), torch.arange(5, M, 30011)]).cuda()
    rows = [out[0].view(torch.uint8)[at].view(F8["e4m3"])] + [o[at] for o in out[1:]]
    check_forward(x[at].cpu(), r[at].cpu(), w.cpu(), rows, "e4m3", False, 1e-6, "bf16")
    h, rstd = out[2], out[3]
    dx, dw = binding.rms_backward(dy, h, w, rstd)
    check_backward(dy[at].cpu(), h[at].cpu(), w.cpu(), rstd[at].cpu(), None, dx[at],
                   torch.from_numpy(R.rms_backward(*(v.double().cpu().numpy() for v in (dy[at], h[at], w, rstd[at])), None)[1]), "bf16")
    terms = dy.double() * h.double() * rstd.double()[:, None]
    # fp32 chains: each of 1536 groups adds its M / 1536 rows in turn, then their sums, two roundings a term
    chain = -(-M // 1536) + 1536 / 64 + 64 + 4
    bound = terms.abs().sum(0) * chain * R.U
    assert bool(((dw.double() - terms.sum(0)).abs() <= bound).all())


def test_norm_of_one_tensor_in_several_places():
    M, D = 700, 1032
    t, _, w = inputs(M, D, "bf16", "bf16", False)
    x, w = t.cuda(), w.cuda()
    want = binding.rms_fp8(x, w, residual=x.clone())
    same = x.clone()
    got = binding.rms_fp8(same, w, residual=same, h_out=same)                # x + x, in its own place
    assert all(same_bits(a, b) for a, b in zip(got, want)) and got[2] is same
    copy = torch.full_like(x, float("nan"))
    got = binding.rms_fp8(x, w, h_out=copy)                                  # no residual: h is a copy of x
    plain = binding.rms_fp8(x, w)
    assert all(same_bits(a, b) for a, b in zip(got, plain)) and same_bits(copy, x)
    for rows in (40, 600, M):                                                # dy, h, dh and dx in one place
        h, rstd = x[:rows], plain[3][:rows]
        want = binding.rms_backward(h.clone(), h.clone(), w, rstd, dh=h.clone())
        one = h.clone()
        got = binding.rms_backward(one, one, w, rstd, dh=one, dx_out=one)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_every_operator_on_another_stream():
    """On a stream or its raw handle, while the current stream is busy with something else."""
    M, D, N = 300, 520, 200
    t, r, w = inputs(M, D, "bf16", "bf16", True)
    x, r, w = t.cuda(), r.cuda(), w.cuda()
    weight = torch.from_numpy(values(np.random.default_rng(3), N, D)).cuda()

    def layer(**kw):
        wq, ws = binding.quantize_fp8(weight, block="tile", **kw)
        q, s, h, rstd = binding.rms_fp8(x, w, residual=r, **kw)
        return binding.run_fp8(q, s, wq, ws, **kw), *binding.rms_backward(x, h, w, rstd, dh=r, **kw)

    want = layer()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.randn((4096, 4096), device="cuda")
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        for _ in range(20):
            busy = busy * 0.5 + 1.0
        got = layer(stream=stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        torch.cuda.synchronize()


def test_two_graphs_of_the_product_and_the_quantiser_in_one_pool():
    """Graphs of one pool replayed in turn, between eager calls that allocate."""
    M, N, K = 130, 200, 400
    rng = np.random.default_rng(9)
    x, y = (torch.from_numpy(values(rng, n, K)).cuda() for n in (M, N))

    def both():
        a, sa = binding.quantize_fp8(x)
        b, sb, bt, sbt = binding.quantize_fp8(y, block="tile", transpose=True)
        return binding.run_fp8(a, sa, b, sb), bt.view(torch.uint8), sbt

    both()
    torch.cuda.synchronize()
    graphs, pool = [], None
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            out = both()
        pool = g.pool()
        graphs.append((g, out))
    for i in range(4):
        x.mul_(-1.5)
        y.copy_(torch.roll(y, 1, 0))
        for g, out in graphs:
            want = both()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))


ONE_EAGER_CALL = """
import torch
from software_pipelined_tiled_02_amd import binding
x, r = (torch.randn((700, 520), device="cuda").bfloat16() for _ in range(2))
w, weight = torch.ones(520, device="cuda").bfloat16(), torch.randn((200, 520), device="cuda")

def layer():
    wq, ws = binding.quantize_fp8(weight, block="tile")
    q, s, h, rstd = binding.rms_fp8(x, w, residual=r)
    return (binding.run_fp8(q, s, wq, ws), binding.run_fp8(q, s, wq, ws, out_dtype=torch.float32, tile="64x64"),
            *binding.rms_backward(x, h, w, rstd, dh=r))

binding.quantize_fp8(torch.ones((4, 256), device="cuda"))
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = layer()
for i in range(3):
    x.mul_(-1.5)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, layer()))
print("captured at first use")
"""


def test_operators_captured_at_their_first_use():
    """One eager call sets the device up; every other operator may meet a capture first."""
    r = subprocess.run([sys.executable, "-c", ONE_EAGER_CALL], cwd=ROOT, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "captured at first use" in r.stdout, r.stdout + r.stderr
