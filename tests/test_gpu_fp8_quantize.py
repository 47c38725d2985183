"""gemm_quantize_fp8 on the GPU: the definition's fp32 operations give the same
bits, so values and scales are compared exactly."""
import numpy as np
import pytest
import torch

from software_pipelined_tiled_02_amd import binding
from tests import fp8_ref as R
from tests.fp8_util import F8, FT, raw_of, values

pytestmark = pytest.mark.gpu


def source(rng, M, K, x):
    t = torch.from_numpy(values(rng, M, K)).to(FT[x])
    return t, t.float().numpy()


def same(q, s, x32, fp8, rows, pow2, what):
    ref, scales = R.quantize_fp32(x32, fp8, rows, pow2)
    assert np.array_equal(s.cpu().numpy(), scales, equal_nan=True), what
    got = raw_of(q)
    nan = np.isnan(R.decode(ref, fp8))
    assert np.array_equal(np.isnan(R.decode(got, fp8)), nan), what
    assert np.array_equal(got[~nan], ref[~nan]), what


@pytest.mark.parametrize("x", ("bf16", "f16", "f32"))
@pytest.mark.parametrize("fp8", ("e4m3", "e5m2"))
@pytest.mark.parametrize("block", ("row", "tile"))
def test_types_blocks_and_directions(x, fp8, block):
    rows = binding.BLOCK_ROWS[block]
    for M, K in ((1, 1), (1, 128), (3, 200), (16, 131), (130, 257), (257, 384), (128, 128)):
        rng = np.random.default_rng(M + K)
        t, x32 = source(rng, M, K, x)
        for pow2 in (False, True):
            q, s = binding.quantize_fp8(t.cuda(), block=block, fp8=fp8, pow2=pow2)
            same(q, s, x32, fp8, rows, pow2, "%dx%d" % (M, K))
            q2, s2, qt, st = binding.quantize_fp8(t.cuda(), block=block, fp8=F8[fp8], pow2=pow2, transpose=True)
            same(q2, s2, x32, fp8, rows, pow2, "%dx%d with transpose" % (M, K))
            same(qt, st, np.ascontiguousarray(x32.T), fp8, rows, pow2, "%dx%d transposed" % (M, K))
            qt2, st2 = binding.quantize_fp8(t.cuda(), block=block, fp8=fp8, pow2=pow2, rows=False, transpose=True)
            assert np.array_equal(raw_of(qt2), raw_of(qt)) and torch.equal(st2, st)
    assert q.stride(0) % 16 == 0 and qt.stride(0) % 16 == 0


@pytest.mark.parametrize("M,K", ((2000, 1100), (5000, 130), (40, 9000)))
def test_many_rows(M, K):
    rng = np.random.default_rng(M)
    t, x32 = source(rng, M, K, "bf16")
    q, s = binding.quantize_fp8(t.cuda())
    same(q, s, x32, "e4m3", 1, False, "rows")
    q, s, qt, st = binding.quantize_fp8(t.cuda(), fp8="e5m2", transpose=True)
    same(q, s, x32, "e5m2", 1, False, "rows")
    same(qt, st, np.ascontiguousarray(x32.T), "e5m2", 1, False, "columns")


def test_borders_zeros_and_what_is_not_finite():
    x = np.zeros((8, 256), dtype=np.float32)
    x[1, 5], x[1, 6] = 1.0, -0.0
    x[2, :128] = np.linspace(-448, 448, 128)                        # scale 1: values on and between steps
    x[3, 7], x[3, 8] = np.nan, 2.0
    x[4, 9], x[4, 10] = np.inf, 3.0
    x[5, 11] = -np.inf
    x[6, 12], x[6, 13] = 1e-45, 1e-40                               # subnormals: the smallest scale
    x[7, 14], x[7, 15] = 3.4028235e38, -1e38                        # the largest fp32
    for fp8 in ("e4m3", "e5m2"):
        for pow2 in (False, True):
            q, s, qt, st = binding.quantize_fp8(torch.from_numpy(x).cuda(), fp8=fp8, pow2=pow2, transpose=True)
            same(q, s, x, fp8, 1, pow2, "rows")
            same(qt, st, np.ascontiguousarray(x.T), fp8, 1, pow2, "columns")
            q, s = binding.quantize_fp8(torch.from_numpy(x).cuda(), fp8=fp8, pow2=pow2, block="tile")
            same(q, s, x, fp8, 128, pow2, "tile")
    v = R.decode(raw_of(binding.quantize_fp8(torch.from_numpy(x).cuda())[0]), "e4m3")
    assert (v[0] == 0).all() and v[1, 5] == 448 and np.isnan(v[3, 7]) and v[3, 8] == 448 and np.isnan(v[4, 9])
    assert v[4, 10] == 0


def test_every_fp32_near_a_step_rounds_to_nearest_even():
    v = R._table("e4m3")[0]
    mid = ((v[1:] + v[:-1]) / 2).astype(np.float32)
    near = np.concatenate([mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9)), v.astype(np.float32)])
    x = np.zeros((len(near), 128), dtype=np.float32)
    x[:, 0], x[:, 1], x[:, 2] = 448.0, near, -near                   # scale 1
    q, s = binding.quantize_fp8(torch.from_numpy(x).cuda())
    same(q, s, x, "e4m3", 1, False, "steps")
    assert bool((s == 1).all())


@pytest.mark.parametrize("ld,offset", ((0, 1), (3, 0), (8, 8), (1, 5)))
def test_rows_at_any_address_and_nothing_else_written(ld, offset):
    """Inputs of any alignment with NaNs between the rows; outputs into a larger
    buffer, of which only the rows change."""
    M, K = 35, 140
    rng = np.random.default_rng(ld + offset)
    g = binding.Gemm(0)
    for x in ("bf16", "f32"):
        t, x32 = source(rng, M, K, x)
        flat = torch.full((offset + M * (K + ld),), float("nan"), dtype=FT[x])
        flat[offset:].as_strided((M, K), (K + ld, 1)).copy_(t)
        src = flat.cuda()[offset:].as_strided((M, K), (K + ld, 1))
        q, s = binding.quantize_fp8(src)
        same(q, s, x32, "e4m3", 1, False, "strided")
        for rows in (1, 128):
            ldq, ldqt, nb, mb = K + ld, M + ld, 2, 1
            qb = torch.full((offset + (M + 1) * ldq,), 0x55, dtype=torch.uint8, device="cuda")
            tb = torch.full((offset + (K + 1) * ldqt,), 0x55, dtype=torch.uint8, device="cuda")
            sb, stb = torch.full((M + 1, nb + 1), 9.0, device="cuda"), torch.full((K + 1, mb + 1), 9.0, device="cuda")
            binding.gemm_quantize_fp8(g.h, M, K, x, "e4m3", rows, 0, src, K + ld, qb.data_ptr() + offset, ldq, sb, nb + 1,
                                      1, tb.data_ptr() + offset, ldqt, stb, mb + 1, 1)
            qv, tv = qb[offset:].as_strided((M, K), (ldq, 1)), tb[offset:].as_strided((K, M), (ldqt, 1))
            n, nt = (M, K) if rows == 1 else (1, nb)
            same(qv, sb[:n, :nb], x32, "e4m3", rows, False, "q")
            same(tv, stb[:nt, :mb], np.ascontiguousarray(x32.T), "e4m3", rows, False, "qt")
            qv.fill_(0x55), tv.fill_(0x55)
            sb[:n, :nb], stb[:nt, :mb] = 9.0, 9.0
            assert bool((qb == 0x55).all()) and bool((tb == 0x55).all())
            assert bool((sb == 9).all()) and bool((stb == 9).all())


def test_offsets_past_32_bits():
    M, K, ld = 9000, 130, 1 << 18
    x = torch.empty((M, ld), dtype=torch.bfloat16, device="cuda")[:, :K]        # 4.7 GB
    x.copy_(torch.randn((M, K), device="cuda"))
    x32 = x.float().cpu().numpy()
    q, s, qt, st = binding.quantize_fp8(x, transpose=True)
    same(q, s, x32, "e4m3", 1, False, "rows")
    same(qt, st, np.ascontiguousarray(x32.T), "e4m3", 1, False, "columns")


def test_sizes_of_zero():
    for M, K in ((0, 5), (5, 0)):
        q, s, qt, st = binding.quantize_fp8(torch.empty((M, K), device="cuda"), transpose=True)
        assert q.shape == (M, K) and qt.shape == (K, M) and s.shape == (M, -(-K // 128)) and st.shape == (K, -(-M // 128))
    torch.cuda.synchronize()


def test_refusals():
    x = torch.zeros((4, 256), device="cuda")
    for call in (lambda: binding.quantize_fp8(x.t()), lambda: binding.quantize_fp8(x[0]),
                 lambda: binding.quantize_fp8(x.double()), lambda: binding.quantize_fp8(x, block="column"),
                 lambda: binding.quantize_fp8(x, fp8="e3m4"), lambda: binding.quantize_fp8(x, rows=False),
                 lambda: binding.quantize_fp8(x[:1].expand(4, 256))):
        with pytest.raises(ValueError):
            call()
