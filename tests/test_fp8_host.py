"""The 8-bit operators on the CPU: the 64-bit reference against hand-checked
values and torch's conversions, and every refusal of the C entry points and of
the binding (all of them before any HIP call)."""
import ctypes

import numpy as np
import pytest
import torch

from software_pipelined_tiled_02_amd import binding
from tests import fp8_ref as R

BAD, ALIGN, UNSUP, OK = (binding.GEMM_ERR_INVALID_ARG, binding.GEMM_ERR_ALIGNMENT, binding.GEMM_ERR_UNSUPPORTED,
                         binding.GEMM_OK)
TORCH = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


# ---- the reference ----------------------------------------------------------

@pytest.mark.parametrize("fp8", ("e4m3", "e5m2"))
def test_decode_is_torchs_for_every_bit_pattern(fp8):
    raw = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(raw).view(TORCH[fp8]).double().numpy()
    assert np.array_equal(R.decode(raw, fp8), t, equal_nan=True)
    assert R.decode([0x38 if fp8 == "e4m3" else 0x3C], fp8)[0] == 1.0


@pytest.mark.parametrize("fp8", ("e4m3", "e5m2"))
def test_encode_is_torchs(fp8):
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(20000) * np.exp2(rng.integers(-20, 8, 20000)),
                        R._table(fp8)[0], -R._table(fp8)[0],
                        (R._table(fp8)[0][1:] + R._table(fp8)[0][:-1]) / 2])      # ties
    x = np.clip(x, -R.TOP[fp8], R.TOP[fp8]).astype(np.float32)
    t = torch.from_numpy(x).to(TORCH[fp8]).view(torch.uint8).numpy()
    assert np.array_equal(R.encode(x.astype(np.float64), fp8), t)


def test_quantize_by_hand():
    x = np.zeros((2, 200), dtype=np.float32)
    x[0, 3], x[0, 4], x[0, 130] = 448.0, -224.0, 1.0
    q, s = R.quantize_fp32(x, "e4m3", 1)
    assert s.shape == (2, 2) and s[0, 0] == 1.0 and s[0, 1] == np.float32(1 / 448.0) and s[1, 0] == np.float32(2.0 ** -126)
    v = R.decode(q, "e4m3")
    assert v[0, 3] == 448 and v[0, 4] == -224 and v[0, 130] == 448 and (v[1] == 0).all()
    q, s = R.quantize_fp32(x, "e4m3", 128, pow2=True)
    assert s.shape == (1, 2) and s[0, 0] == 1.0 and s[0, 1] == 2.0 ** -8
    assert R.decode(q, "e4m3")[0, 130] == 256


def test_product_by_hand():
    a, b = np.zeros((1, 256)), np.zeros((2, 256))
    a[0, 0], a[0, 200] = 2.0, 3.0
    b[1, 0], b[1, 200] = 5.0, 7.0
    C, _, _ = R.product(a, np.array([[10.0, 100.0]]), b, np.array([[1.0, 2.0]]), 128)
    assert C[0, 0] == 0 and C[0, 1] == 2 * 5 * 10 + 3 * 7 * 200
    C, _, _ = R.product(a, np.array([[10.0, 100.0]]), b, np.array([[1.0, 2.0], [0.5, 0.25]]), 1)
    assert C[0, 1] == 2 * 5 * 5 + 3 * 7 * 25


@pytest.mark.parametrize("with_dh", (False, True))
def test_rms_backward_is_the_forwards_derivative(with_dh):
    """The backward formula against central differences of the forward one, in 64 bits."""
    rng = np.random.default_rng(2)
    M, D, eps = 3, 37, 1e-3
    h, w, dy = rng.standard_normal((M, D)), rng.standard_normal(D), rng.standard_normal((M, D))
    dh = rng.standard_normal((M, D)) if with_dh else None

    def loss(h, w):
        return (R.rms(h, None, w, eps)[0] * dy).sum() + ((h * dh).sum() if with_dh else 0.0)

    dx, dw = R.rms_backward(dy, h, w, R.rms(h, None, w, eps)[1], dh)
    step = 1e-5      # truncation ~ step^2, rounding ~ 1e-16 * |loss| / step: both below 1e-9
    for i, j in ((0, 0), (1, 17), (2, 36)):
        d = np.zeros_like(h)
        d[i, j] = step
        assert abs((loss(h + d, w) - loss(h - d, w)) / (2 * step) - dx[i, j]) < 1e-8
    for j in (0, 20):
        d = np.zeros_like(w)
        d[j] = step
        assert abs((loss(h, w + d) - loss(h, w - d)) / (2 * step) - dw[j]) < 1e-8


# ---- the product's plan and refusals ----------------------------------------

def q(M=512, N=512, K=512, **kw):
    return binding.gemm_query_fp8(M, N, K, check=False, **kw)


def test_product_plan():
    """The class that takes the least time by the measured costs, for 256 CUs."""
    T = binding.FP8_TILES
    for M, N, K, tile in ((1, 4096, 4096, "16x16"), (16, 4096, 8192, "16x16"), (1, 8192, 8192, "16x32"), (32, 8192, 8192, "64x32"),
                          (64, 8192, 8192, "64x32"), (128, 4096, 4096, "64x32"), (256, 4096, 4096, "64x64k4"), (512, 4096, 4096, "64x64"),
                          (500, 4104, 4100, "128x128"), (1024, 4096, 4096, "128x128"), (2048, 4096, 4096, "256x128"),
                          (4096, 4096, 4096, "256x256"), (8192, 8192, 8200, "256x256"), (0, 16, 16, None),
                          (16, 16, 0, None)):
        rc, info = q(M, N, K)
        assert rc == OK and (tile is None or info["tile"] == T[tile]), (M, N, K, info)
        assert info["c_tiles"] == -(-M // info["block_m"]) * -(-N // info["block_n"])
        assert info["grid"] == min(info["c_tiles"], 256 if tile == "256x256" else 1 << 31)
        assert info["k_blocks"] == -(-K // 128)
    assert q(4096, 4096, 4096, c_dtype="f32")[1]["tile"] == T["256x128"]       # fp32 outputs: widened
    assert q(4096, 4096, 4096, c_dtype="f32")[1]["widened"] == 1
    assert q(1, 8192, 8192, c_dtype="f32")[1]["tile"] == T["16x32"]
    assert q(4096, 4096, 4100, lda=4100)[1]["staged"] == 0                      # rows at any address
    assert q(4096, 4096, 4100, A=8)[1]["staged"] == 0
    assert q(4096, 4096, 4100)[1]["staged"] == 1                                # any K with rows on 16 bytes


def test_product_refusals():
    assert q(a_type=1)[0] == BAD and q(b_type=18)[0] == BAD and q(c_dtype="i8")[0] == BAD
    assert q(b_scale_rows=64)[0] == BAD and q(tile=9)[0] == BAD and q(tile=-2)[0] == BAD
    assert q(accumulate=2)[0] == BAD and q(accumulate=1)[0] == UNSUP
    assert q(accumulate=1, c_dtype="f32")[0] == OK
    assert q(M=-1)[0] == BAD and q(N=-1)[0] == BAD and q(K=-1)[0] == BAD
    assert q(lda=511)[0] == BAD and q(ldb=511)[0] == BAD and q(ldc=511)[0] == BAD
    assert q(sa_row=-1)[0] == BAD and q(sb_blk=-1)[0] == BAD
    assert q(C=1)[0] == ALIGN and q(SA=2)[0] == ALIGN and q(SB=6)[0] == ALIGN
    assert q(C=2)[0] == OK and q(C=2, c_dtype="f32")[0] == ALIGN
    assert q(tile="256x256", lda=520)[0] == ALIGN                               # rows not on 16 bytes
    assert q(tile="256x256", c_dtype="f32")[0] == UNSUP
    assert q(K=2 ** 31 - 1, lda=2 ** 31)[0] == UNSUP
    assert q(lda=1 << 28)[0] == UNSUP and q(ldb=1 << 28)[0] == UNSUP            # a tile's rows: 2^31 bytes
    assert q(sa_row=1 << 24)[0] == UNSUP and q(sb_blk=1 << 28)[0] == UNSUP      # a tile's, a row's scales
    assert q(sa_row=0, sa_blk=0, sb_row=0, sb_blk=0)[0] == OK                   # expanded scales
    assert q(M=0)[0] == OK and q(N=0)[0] == OK and q(K=0)[0] == OK and q(K=0, tile="128x128")[0] == OK
    assert q(M=0)[1]["grid"] == 0
    rc = binding.gemm_run_fp8(None, 16, 16, 16, "e4m3", "e4m3", "bf16", 128, 0, "auto", 0, 16, 0, 1, 16, 0, 16, 0, 1, 1,
                              0, 16, stream=0, check=False)
    assert rc == BAD
    with pytest.raises(binding.GemmError):
        binding.gemm_query_fp8(16, 16, 16, lda=8)


def test_product_refuses_scales_past_the_buffers_range():
    """A scale's address is the sum of its row's and its block's parts, which has to stay below 2^31
    bytes (a load past it gives zero): both sides of the border, of A's and of B's scales."""
    far = dict(M=256, N=256, K=256, tile="256x256")
    assert q(sa_row=2 ** 21 - 1, sa_blk=2 ** 28 - 1, **far)[0] == UNSUP         # row 255, block 1: 3.2 GB
    assert q(sa_row=2 ** 20, sa_blk=2 ** 27 - 1, **far)[0] == OK                # 256 rows and 2 blocks: 2^31 - 8
    assert q(sa_row=2 ** 20, sa_blk=2 ** 27, **far)[0] == UNSUP
    rows = dict(far, b_scale_rows=1)
    assert q(sb_row=2 ** 20, sb_blk=2 ** 27 - 1, **rows)[0] == OK
    assert q(sb_row=2 ** 20, sb_blk=2 ** 27, **rows)[0] == UNSUP
    assert q(sb_row=2 ** 27, sb_blk=2 ** 27 - 1, **far)[0] == OK                # tiles: two rows of scales
    assert q(sb_row=2 ** 27, sb_blk=2 ** 27, **far)[0] == UNSUP
    assert q(sa_row=2 ** 62, sa_blk=2 ** 62, **far)[0] == UNSUP                 # (no overflow in the check)
    assert q(M=1, N=256, K=128, sa_row=2 ** 62, sa_blk=2 ** 62)[0] == OK        # one scale: no stride counts


def test_product_refuses_rows_whose_offsets_leave_32_bits():
    """The loops address up to 16 blocks past K, out of range by a bit of their own: the rows' span
    leaves room for them.  Both sides of the border, of A and of B."""
    far = dict(M=32, N=32, tile="32x32", sa_blk=1, sb_blk=1)
    assert q(K=2 ** 26 - 16, lda=2 ** 26 - 16, ldb=2 ** 26 - 16, **far)[0] == UNSUP
    assert q(K=2 ** 26 - 128, lda=2 ** 26 - 128, ldb=2 ** 26 - 128, **far)[0] == OK
    assert q(K=2 ** 26 - 128, lda=2 ** 26 - 112, ldb=2 ** 26 - 128, **far)[0] == UNSUP
    assert q(K=2 ** 26 - 128, lda=2 ** 26 - 128, ldb=2 ** 26 - 112, **far)[0] == UNSUP
    one = dict(M=1, N=1, tile="16x16", lda=2 ** 62, ldb=2 ** 62)                # one row: its K counts
    assert q(K=2 ** 31 - 4096, **one)[0] == OK and q(K=2 ** 31 - 4095, **one)[0] == UNSUP


@pytest.mark.parametrize("size", ((4096, 4096, 4096), (512, 512, 512), (64, 8192, 8192), (5, 4096, 4096), (8192, 8192, 8200)))
def test_auto_takes_what_some_class_takes(size):
    """Strides too wide for the cheapest class go to the next one that reaches."""
    M, N, K = size
    wide = [dict(lda=1 << e) for e in range(14, 31)] + [dict(ldb=1 << e) for e in range(14, 31)]
    wide += [dict(sa_row=1 << e, sa_blk=1) for e in range(10, 30)] + [dict(sb_row=1 << e, sb_blk=1) for e in range(10, 30)]
    wide += [dict(b_scale_rows=1, sb_row=1 << e, sb_blk=1) for e in range(10, 30)]
    for kw in wide:
        rc, info = q(M, N, K, **kw)
        takes = [t for t in range(9) if q(M, N, K, tile=t, **kw)[0] == OK]
        if any(t <= 6 for t in takes) or (M <= 32 and takes):
            assert rc == OK and info["tile"] in takes, (kw, takes)
        elif not takes:
            assert rc == UNSUP, kw
    assert q(4096, 4096, 4096, lda=1 << 23)[1]["tile"] == binding.FP8_TILES["128x128"]
    assert q(4096, 4096, 4096, sa_row=1 << 21, sa_blk=1)[0] == OK
    assert q(4096, 4096, 4096)[1]["tile"] == binding.FP8_TILES["256x256"]


class FakeHandle:
    """Enough of a handle for calls that are refused before it is used: the
    entry points check every argument before any HIP call.  (Device 0 with 256
    CUs: the first two integers.)"""

    def __init__(self):
        self.block = (ctypes.c_int * 16)(0, 256)
        self.h = ctypes.addressof(self.block)


FAKE = FakeHandle()
H = FAKE.h
P = 4096                   # an aligned address; refused calls never read it


def run(**kw):
    a = dict(M=512, N=512, K=512, a="e4m3", b="e4m3", c="bf16", rows=128, acc=0, tile="auto", A=P, lda=512, SA=P,
             sa_row=1, sa_blk=512, B=P, ldb=512, SB=P, sb_row=1, sb_blk=4, C=P, ldc=512)
    a.update(kw)
    return binding.gemm_run_fp8(H, *a.values(), stream=0, check=False)


def test_product_null_pointers():
    for name in ("A", "B", "SA", "SB", "C"):
        assert run(**{name: None}) == BAD, name
    assert run(K=0, A=None, B=None, SA=None, SB=None, C=None) == BAD            # C = 0 has to go somewhere
    for zero in ("M", "N"):
        assert run(**{zero: 0, "A": None, "B": None, "SA": None, "SB": None, "C": None}) == OK


def quant(**kw):
    a = dict(M=256, K=256, x="bf16", f="e4m3", rows=1, pow2=0, X=P, ldx=256, Q=P, ldq=256, S=P, s_row=1, s_blk=256,
             QT=P, ldqt=256, ST=P, st_row=1, st_blk=256)
    a.update(kw)
    return binding.gemm_quantize_fp8(H, *a.values(), stream=0, check=False)


def test_quantize_refusals():
    assert quant(x="i8") == BAD and quant(f=0) == BAD and quant(rows=2) == BAD and quant(pow2=2) == BAD
    assert quant(M=-1) == BAD and quant(K=-1) == BAD and quant(s_row=-1) == BAD and quant(st_blk=-1) == BAD
    assert quant(ldx=255) == BAD and quant(ldq=255) == BAD and quant(ldqt=255) == BAD
    assert quant(X=None) == BAD and quant(S=None) == BAD and quant(ST=None) == BAD
    assert quant(Q=None, QT=None) == BAD
    assert quant(X=P + 1) == ALIGN and quant(S=P + 2) == ALIGN and quant(x="f32", X=P + 2) == ALIGN
    assert quant(M=2 ** 31, ldqt=2 ** 31) == UNSUP
    assert quant(M=2 ** 30, K=2 ** 14, ldx=2 ** 14, ldq=2 ** 14, ldqt=2 ** 30) == UNSUP     # 2^30 workgroups
    assert quant(M=0, X=None) == OK and quant(K=0, X=None) == OK
    assert binding.gemm_quantize_fp8(None, 1, 1, "bf16", "e4m3", 1, 0, P, 1, P, 1, P, 1, 1, stream=0, check=False) == BAD


def test_quantize_refuses_launches_of_too_many_threads():
    """A launch takes less than 2^32 threads: 2^24 workgroups of 256, or 2^23 of 512."""
    M = 2 ** 30 - 127                                                           # 2^23 row blocks of 128
    one = dict(K=1, ldx=1, ldq=1, s_blk=M, ldqt=M, st_blk=1)
    assert quant(M=M, **one) == UNSUP and quant(M=M, rows=128, **one) == UNSUP
    assert quant(M=M, rows=128, **dict(one, QT=None)) == UNSUP
    wide = dict(K=2 ** 30 - 127, M=128, ldx=2 ** 30, ldq=2 ** 30, ldqt=128)     # 2^23 column blocks of 128
    assert quant(rows=128, **wide) == UNSUP and quant(**wide) == UNSUP
    assert quant(M=2 ** 30 - 63, K=1, QT=None) == UNSUP                         # rows alone: 2^24 of 64


def rms(**kw):
    a = dict(M=4, D=256, x="bf16", w="bf16", f="e4m3", pow2=0, eps=1e-6, X=P, ldx=256, R=P, ldr=256, W=P, H=P, ldh=256,
             Y=P, ldy=256, Q=P, ldq=256, S=P, s_row=1, s_blk=4, rstd=P)
    a.update(kw)
    return binding.gemm_rms_fp8(H, *a.values(), stream=0, check=False)


def test_rms_refusals():
    assert rms(x="i8") == BAD and rms(w="f16") == BAD and rms(f=3) == BAD and rms(pow2=-1) == BAD
    assert rms(eps=-1.0) == BAD and rms(eps=float("nan")) == BAD
    assert rms(M=-1) == BAD and rms(D=-1) == BAD and rms(s_row=-1) == BAD
    for ld in ("ldx", "ldr", "ldh", "ldy", "ldq"):
        assert rms(**{ld: 255}) == BAD, ld
    assert rms(X=None) == BAD and rms(W=None) == BAD and rms(S=None) == BAD and rms(Q=None, Y=None) == BAD
    for p in ("X", "R", "H", "Y", "W"):
        assert rms(**{p: P + 1}) == ALIGN, p
    assert rms(S=P + 2) == ALIGN and rms(rstd=P + 2) == ALIGN and rms(w="f32", W=P + 2) == ALIGN
    big = binding.GEMM_RMS_MAX_D + 1
    assert rms(D=big, ldx=big, ldr=big, ldh=big, ldy=big, ldq=big) == UNSUP
    assert rms(M=binding.GEMM_RMS_MAX_ROWS + 1) == UNSUP
    assert rms(M=0, X=None, W=None) == OK and rms(D=0, X=None) == OK


def rms_back(**kw):
    a = dict(M=4, D=256, x="bf16", w="f32", DY=P, lddy=256, Hm=P, ldh=256, W=P, rstd=P, DH=P, lddh=256, DX=P, lddx=256,
             DW=P, ws=P, nbytes=1 << 20)
    a.update(kw)
    return binding.gemm_rms_backward(H, *a.values(), stream=0, check=False)


def test_rms_backward_refusals():
    assert rms_back(x="i8") == BAD and rms_back(w="f16") == BAD and rms_back(M=-1) == BAD and rms_back(D=-1) == BAD
    for ld in ("lddy", "ldh", "lddh", "lddx"):
        assert rms_back(**{ld: 255}) == BAD, ld
    for p in ("DY", "Hm", "W", "rstd", "DX", "DW"):
        assert rms_back(**{p: None}) == BAD, p
    need = binding.gemm_rms_backward_workspace(4096, 256)
    assert rms_back(M=4096, ws=None) == BAD and rms_back(M=4096, nbytes=need - 1) == BAD and rms_back(nbytes=-1) == BAD
    for p in ("DY", "Hm", "DH", "DX"):
        assert rms_back(**{p: P + 1}) == ALIGN, p
    assert rms_back(ws=P + 8) == ALIGN and rms_back(DW=P + 2) == ALIGN
    assert rms_back(M=binding.GEMM_RMS_MAX_ROWS + 1) == UNSUP
    big = binding.GEMM_RMS_MAX_D + 1
    assert rms_back(D=big, lddy=big, ldh=big, lddh=big, lddx=big) == UNSUP
    assert rms_back(D=0, DW=None) == OK


def test_rms_refuses_launches_of_too_many_threads():
    """A launch takes less than 2^32 threads; long rows have 1024 each."""
    M = binding.GEMM_RMS_MAX_ROWS
    for D in (8193, 8200, 16384, 32768):
        assert rms(M=M, D=D, ldx=D, ldr=D, ldh=D, ldy=D, ldq=D) == UNSUP, D
    for D in (12289, 16385, 32768):
        for rows in (M, M - 1):                          # the columns of dw take workgroups too
            assert rms_back(M=rows, D=D, lddy=D, ldh=D, lddh=D, lddx=D, nbytes=1 << 30) == UNSUP, D
    assert rms_back(M=M - 16384, D=32768, lddy=32768, ldh=32768, lddh=32768, lddx=32768, nbytes=1 << 30) == UNSUP


def test_rms_backward_workspace():
    ws = binding.gemm_rms_backward_workspace
    assert ws(4, 256) == ws(512, 8192) == ws(0, 256) == 0                       # few rows: none
    assert ws(513, 2048) % (2048 * 4) == 0 and ws(513, 2046) == ws(513, 2048) > 0
    assert ws(-1, 256) == 0 and ws(1, binding.GEMM_RMS_MAX_D + 1) == 0
    assert ws(1 << 20, 8192) == ws(1 << 21, 8192) > 0                           # bounded
    assert ws(1 << 20, 20000) == ws(1 << 21, 20000) > 0


# ---- the torch functions' refusals (CPU tensors: nothing is enqueued) --------

def test_binding_refuses_what_is_no_device_matrix():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    q8 = torch.zeros(4, 256, dtype=torch.float8_e4m3fn)
    s = torch.ones(4, 2)
    for call in (lambda: binding.run_fp8(q8, s, q8, s), lambda: binding.run_fp8(x, s, q8, s),
                 lambda: binding.run_fp8([1], s, q8, s), lambda: binding.run_fp8(q8[0], s, q8, s),
                 lambda: binding.quantize_fp8(x), lambda: binding.quantize_fp8(x.to(torch.int8)),
                 lambda: binding.quantize_fp8(None), lambda: binding.rms_fp8(x, x[0]),
                 lambda: binding.rms_fp8(x[0], x[0]), lambda: binding.rms_backward(x, x, x[0], s[:, 0])):
        with pytest.raises(ValueError):
            call()
