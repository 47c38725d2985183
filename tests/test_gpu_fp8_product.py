"""gemm_run_fp8 on the GPU against its definition in 64 bits (fp8_ref states the bounds)."""
import numpy as np
import pytest
import torch

from software_pipelined_tiled_02_amd import binding
from tests import fp8_ref as R
from tests.fp8_util import F8, FT, check_product, f8_of, operand, place_bytes, run_product

pytestmark = pytest.mark.gpu

TILES = ("256x256", "256x128", "128x128", "64x64", "64x64k4", "64x32", "32x32", "16x32", "16x16")


def case(M, N, K, at="e4m3", bt="e4m3", rows=128, seed=0):
    rng = np.random.default_rng(seed + 7 * M + 3 * N + K)
    a, sa = operand(rng, M, K, at, 1)
    b, sb = operand(rng, N, K, bt, rows)
    return a, sa, b, sb


@pytest.mark.parametrize("out", ("bf16", "f16", "f32"))
@pytest.mark.parametrize("rows", (128, 1))
@pytest.mark.parametrize("tile", TILES)
def test_every_tile(tile, rows, out):
    if tile == "256x256" and out == "f32":
        pytest.skip("refused: fp32 outputs stop at 256x128")
    for M, N, K in ((33, 140, 300), (259, 131, 128), (256, 256, 272), (16, 16, 1040)):
        a, sa, b, sb = case(M, N, K, rows=rows)
        c = run_product(a, sa, b, sb, "e4m3", "e4m3", out_dtype=FT[out], tile=tile)
        check_product(c, a, sa, b, sb, "e4m3", "e4m3", rows, out, "%s %dx%dx%d" % (tile, M, N, K))


@pytest.mark.parametrize("K", (2000, 2176, 3733))
@pytest.mark.parametrize("tile", TILES)
def test_many_blocks(tile, K):
    """Blocks whose share among the waves is even and uneven, rings that are refilled often."""
    for rows, out in ((128, "bf16"), (1, "f32")):
        if tile == "256x256" and out == "f32":
            continue
        a, sa, b, sb = case(70, 65, K, rows=rows)
        c = run_product(a, sa, b, sb, "e4m3", "e4m3", out_dtype=FT[out], tile=tile)
        check_product(c, a, sa, b, sb, "e4m3", "e4m3", rows, out, "%s %d" % (tile, K))


@pytest.mark.parametrize("at,bt", (("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")))
@pytest.mark.parametrize("tile", TILES)
def test_types(tile, at, bt):
    for out in ("bf16", "f32"):
        if tile == "256x256" and out == "f32":
            continue
        a, sa, b, sb = case(70, 150, 270, at, bt, 1 if out == "f32" else 128)
        c = run_product(a, sa, b, sb, at, bt, out_dtype=FT[out], tile=tile)
        check_product(c, a, sa, b, sb, at, bt, 1 if out == "f32" else 128, out, "%s %s %s" % (tile, at, bt))


@pytest.mark.parametrize("M,N,K", ((1, 1, 1), (1, 300, 16), (2, 3, 17), (15, 17, 127), (17, 129, 129), (1, 64, 5000),
                                   (64, 257, 255), (300, 20, 641), (130, 130, 2049)))
def test_auto_sizes(M, N, K):
    for out in ("bf16", "f32"):
        a, sa, b, sb = case(M, N, K)
        c = run_product(a, sa, b, sb, "e4m3", "e4m3", out_dtype=FT[out])
        check_product(c, a, sa, b, sb, "e4m3", "e4m3", 128, out, "%dx%dx%d" % (M, N, K))


def test_every_tile_gives_the_same_sums_of_one_block():
    """K = 128: one instruction per piece, so every tile class gives the same bits."""
    a, sa, b, sb = case(300, 200, 128)
    got = [run_product(a, sa, b, sb, "e4m3", "e4m3", tile=t).view(torch.int16) for t in TILES]
    for g in got[1:]:
        assert torch.equal(g, got[0])


@pytest.mark.parametrize("K", (1, 31, 100, 128, 200, 383))
@pytest.mark.parametrize("lda,offset", ((0, 0), (5, 0), (0, 3), (16, 8), (3, 1)))
def test_rows_at_any_address(K, lda, offset):
    """Bases and row strides of any alignment; the bytes around the rows are NaNs, and
    none follows the last one's end."""
    for M, N in ((5, 33), (70, 70)):
        a, sa, b, sb = case(M, N, K, "e4m3", "e5m2")
        for out in ("f16", "f32"):
            c = binding.run_fp8(place_bytes(a, K + lda, offset).view(F8["e4m3"]), torch.from_numpy(sa).cuda(),
                                place_bytes(b, K + lda + 1, offset + 1).view(F8["e5m2"]), torch.from_numpy(sb).cuda(),
                                out_dtype=FT[out])
            check_product(c, a, sa, b, sb, "e4m3", "e5m2", 128, out, "K=%d +%d @%d" % (K, lda, offset))


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("N,ldc,offset", ((130, 130, 0), (131, 133, 1), (128, 136, 4), (129, 140, 8)))
def test_output_stays_inside_its_rows(tile, N, ldc, offset):
    M, K = 37, 144
    a, sa, b, sb = case(M, N, K)
    for out in ("bf16", "f32"):
        if tile == "256x256" and out == "f32":
            continue
        flat = torch.full((offset + (M + 1) * ldc,), 7.0, dtype=FT[out], device="cuda")
        c = flat[offset:].as_strided((M, N), (ldc, 1))
        assert run_product(a, sa, b, sb, "e4m3", "e4m3", out=c, tile=tile) is c
        check_product(c, a, sa, b, sb, "e4m3", "e4m3", 128, out, tile)
        rest = flat.clone()
        rest[offset:].as_strided((M, N), (ldc, 1)).fill_(7.0)
        assert bool((rest == 7.0).all())


@pytest.mark.parametrize("tile", TILES[1:])
@pytest.mark.parametrize("M,N", ((70, 131), (300, 272)))
def test_accumulate(tile, M, N):
    K = 400
    a, sa, b, sb = case(M, N, K, rows=1)
    c = torch.randn((M, N), device="cuda")
    base = c.double().cpu().numpy()
    run_product(a, sa, b, sb, "e4m3", "e4m3", out=c, accumulate=True, tile=tile)
    check_product(c, a, sa, b, sb, "e4m3", "e4m3", 1, "f32", tile, base)
    c = torch.full((M, N), float("nan"), device="cuda")          # not read without accumulate
    run_product(a, sa, b, sb, "e4m3", "e4m3", out=c, tile=tile)
    check_product(c, a, sa, b, sb, "e4m3", "e4m3", 1, "f32", tile)
    c.fill_(3.0)
    e = torch.empty((M, 0), dtype=F8["e4m3"], device="cuda")
    f = torch.empty((N, 0), dtype=F8["e4m3"], device="cuda")
    none = torch.empty((M, 0), device="cuda"), torch.empty((N, 0), device="cuda")
    binding.run_fp8(e, none[0], f, none[1], out=c, accumulate=True, tile=tile)
    assert bool((c == 3.0).all())
    binding.run_fp8(e, none[0], f, none[1], out=c, tile=tile)
    assert bool((c == 0.0).all())


def test_sizes_of_zero():
    for M, N in ((0, 5), (5, 0), (0, 0)):
        a, b = (torch.empty((n, 256), dtype=F8["e4m3"], device="cuda") for n in (M, N))
        c = binding.run_fp8(a, torch.empty((M, 2), device="cuda"), b, torch.empty((-(-N // 128), 2), device="cuda"))
        assert c.shape == (M, N) and c.dtype == torch.bfloat16
    torch.cuda.synchronize()


@pytest.mark.parametrize("tile", TILES)
def test_no_columns_and_far_rows(tile):
    """K = 0: C is zeros, and the strides of rows and scales without elements do not matter."""
    M, N, ld = 70, 130, 2 ** 31 - 16
    a, b = (torch.empty(0, dtype=F8["e4m3"], device="cuda").as_strided((n, 0), (ld, 1)) for n in (M, N))
    sa, sb = (torch.empty(0, device="cuda").as_strided((n, 0), (2 ** 29 - 1, 2 ** 29 - 1)) for n in (M, 2))
    c = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    binding.run_fp8(a, sa, b, sb, out=c, tile=tile)
    assert bool((c == 0.0).all())


@pytest.mark.parametrize("tile", TILES)
def test_nan_infinity_and_scales(tile):
    """NaNs, infinities (e5m2) and scales of zero, infinity and NaN reach their row and column alone."""
    M, N, K = 20, 140, 272
    a, sa, b, sb = case(M, N, K, "e5m2", "e4m3", 128)
    a[3, 100], a[5, 271], a[7, 0] = 0x7F, 0x7C, 0xFC              # NaN, inf, -inf
    b[9, 271] = 0x7F
    b[12, :] = 0                                                 # zeros: 0 * inf = NaN beside row 5 and 7
    sa[11, 1], sa[13, 0], sa[15, 2] = 0.0, np.inf, np.nan
    c = run_product(a, sa, b, sb, "e5m2", "e4m3", out_dtype=torch.bfloat16, tile=tile)
    check_product(c, a, sa, b, sb, "e5m2", "e4m3", 128, "bf16", tile)
    got = c.float().cpu().numpy()
    assert np.isnan(got[3]).all() and np.isnan(got[:, 9]).all() and np.isnan(got[15]).all() and np.isnan(got[5, 12])
    rows = [i for i in range(M) if i not in (3, 5, 7, 13, 15)]
    assert np.isfinite(got[rows][:, [j for j in range(N) if j != 9]]).all()


@pytest.mark.parametrize("tile", TILES)
def test_extreme_and_subnormal_values(tile):
    """Largest and smallest 8-bit values, subnormals among them."""
    M, N, K = 18, 129, 144
    rng = np.random.default_rng(4)
    pick = np.array([0x7E, 0xFE, 0x01, 0x81, 0x07, 0x08, 0x00, 0x80], dtype=np.uint8)
    a, b = (pick[rng.integers(0, len(pick), (n, K))] for n in (M, N))
    sa, sb = np.ones((M, 2), np.float32), np.full((2, 2), 2.0 ** -20, np.float32)
    for out in ("bf16", "f32"):
        if tile == "256x256" and out == "f32":
            continue
        c = run_product(a, sa, b, sb, "e4m3", "e4m3", out_dtype=FT[out], tile=tile)
        check_product(c, a, sa, b, sb, "e4m3", "e4m3", 128, out, tile)
    a = np.full((M, K), 0x01, dtype=np.uint8)                    # 2^-9 each: no subnormal is lost
    b = np.full((N, K), 0x38, dtype=np.uint8)
    c = run_product(a, sa, b, np.ones_like(sb), "e4m3", "e4m3", out_dtype=FT["bf16"], tile=tile)
    assert bool((c == 144 * 2.0 ** -9).all())


def test_scales_of_any_strides():
    M, N, K = 40, 300, 390
    a, sa, b, sb = case(M, N, K, rows=1)
    at, bt = f8_of(np.pad(a, ((0, 0), (0, 10))), "e4m3")[:, :K], f8_of(np.pad(b, ((0, 0), (0, 10))), "e4m3")[:, :K]
    ref = binding.run_fp8(at, torch.from_numpy(sa).cuda(), bt, torch.from_numpy(sb).cuda())
    wide = torch.full((4, 3, M), float("nan"), device="cuda")
    wide[:, 1] = torch.from_numpy(sa).cuda().t()
    c = binding.run_fp8(at, wide[:, 1].t(), bt, torch.from_numpy(sb).cuda().t().contiguous().t())
    assert torch.equal(c, ref)
    one = torch.full((1, 1), 0.25, device="cuda")                 # one scale for all of A: expanded
    c = binding.run_fp8(at, one.expand(M, 4), bt, one.expand(N, 4))
    check_product(c, a, np.full((M, 4), 0.25, np.float32), b, np.full((N, 4), 0.25, np.float32), "e4m3", "e4m3", 1,
                  "bf16", "expanded")


@pytest.mark.parametrize("tile", ("256x256", "64x64", "64x64k4", "64x32"))
def test_offsets_past_32_bits(tile):
    """Rows of A, B and C more than 2^32 bytes from their base."""
    M, N, K, ld = 33000, 16, 144, 1 << 17
    rng = np.random.default_rng(8)
    rows = np.array([0, 1, 16383, 16384, 32766, 32999])
    a, sa = operand(rng, len(rows), K, "e4m3", 1)
    b, sb = operand(rng, N, K, "e4m3", 128)
    buf = torch.empty((M, ld), dtype=torch.uint8, device="cuda")
    buf[:, :K] = 0
    buf[rows, :K] = torch.from_numpy(a).cuda()
    s = torch.zeros((M, 2), device="cuda")
    s[rows] = torch.from_numpy(sa).cuda()
    c = torch.empty((M, ld // 2), dtype=torch.bfloat16, device="cuda")[:, :N]
    binding.run_fp8(buf.view(F8["e4m3"])[:, :K], s, f8_of(b, "e4m3"), torch.from_numpy(sb).cuda(), out=c, tile=tile)
    check_product(c[rows], a, sa, b, sb, "e4m3", "e4m3", 128, "bf16", tile)
    assert int((c != 0).any(dim=1).sum()) == len(rows)
    if tile == "64x32":                                            # the long matrix as the second factor
        ct = torch.empty((N, M), dtype=torch.bfloat16, device="cuda")
        binding.run_fp8(f8_of(b, "e4m3"), torch.from_numpy(np.repeat(sb, N, 0)).cuda(), buf.view(F8["e4m3"])[:, :K], s,
                        out=ct, tile=tile)
        check_product(ct[:, torch.from_numpy(rows).cuda()], b, np.repeat(sb, N, 0), a, sa, "e4m3", "e4m3", 1, "bf16", tile)


@pytest.mark.parametrize("tile", TILES)
def test_a_very_long_k(tile):
    """Two rows of 2^28 + 20 columns, all but a few of them zero: offsets near the border of what is taken."""
    M, N, K = 1, 2, 2 ** 28 + 20
    at, nb = (0, 2 ** 27 - 1, 2 ** 27, 2 ** 28 - 129, 2 ** 28, K - 1), -(-K // 128)
    a, b = (torch.zeros((n, K + 12), dtype=torch.uint8, device="cuda") for n in (M, N))
    for i, k in enumerate(at):
        a[0, k], b[1, k] = 0x38 + i, 0x40                          # 1 + i / 8 and 2
    b[0, K - 1] = 0x38
    s = torch.ones((1, nb), device="cuda")
    c = binding.run_fp8(a.view(F8["e4m3"])[:, :K], s, b.view(F8["e4m3"])[:, :K], s, tile=tile)
    assert c.tolist() == [[1 + 5 / 8, 2 * (6 + 15 / 8)]]


@pytest.mark.parametrize("tile,rows", (("256x256", 128), ("256x256", 1), ("128x128", 128)))
def test_more_tiles_than_one_round(tile, rows):
    """More than 256 tiles: workgroups take several in turn, and K-tiles start at
    a place that depends on the tile.  Sampled rows and columns, the edges' among them."""
    M, N, K = 4353, 4100, 400
    a, sa, b, sb = case(M, N, K, rows=rows)
    c = run_product(a, sa, b, sb, "e4m3", "e4m3", tile=tile)
    rng = np.random.default_rng(1)
    i = np.unique(np.concatenate([[0, 255, 256, 4095, 4351, 4352], rng.integers(0, M, 60)]))
    j = np.unique(np.concatenate([[0, 127, 128, 255, 256, 4095, 4096, 4099], rng.integers(0, N, 60)]))
    part = c[torch.from_numpy(i).cuda()][:, torch.from_numpy(j).cuda()]
    check_product(part, a[i], sa[i], b[j], np.repeat(sb, rows, 0)[j], "e4m3", "e4m3", 1, "bf16", tile)
    assert torch.equal(c, run_product(a, sa, b, sb, "e4m3", "e4m3", tile=tile))       # the same bits each time


def test_streams_and_reuse_of_freed_memory():
    """A call on another stream: what it allocates belongs to that stream."""
    a, sa, b, sb = case(128, 256, 512)
    args = [f8_of(a, "e4m3"), torch.from_numpy(sa).cuda(), f8_of(b, "e4m3"), torch.from_numpy(sb).cuda()]
    ref = binding.run_fp8(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        got = [binding.run_fp8(*args, stream=stream) for _ in range(8)]
        side.synchronize()
        assert all(torch.equal(g, ref) for g in got)


def test_graph_replays():
    a, sa, b, sb = case(96, 160, 400)
    args = [f8_of(np.pad(a, ((0, 0), (0, 0))), "e4m3"), torch.from_numpy(sa).cuda(), f8_of(b, "e4m3"),
            torch.from_numpy(sb).cuda()]
    binding.run_fp8(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = binding.run_fp8(*args, out_dtype=torch.float32)
    for seed in range(4):
        a2, sa2, b2, sb2 = case(96, 160, 400, seed=seed)
        for t, v in zip(args, (a2, sa2, b2, sb2)):
            t.view(torch.uint8).copy_(torch.from_numpy(np.ascontiguousarray(v)).view(torch.uint8))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, binding.run_fp8(*args, out_dtype=torch.float32))
        check_product(c, a2, sa2, b2, sb2, "e4m3", "e4m3", 128, "f32", "replay %d" % seed)


def test_refusals():
    a = torch.zeros((32, 256), dtype=F8["e4m3"], device="cuda")
    s, s1 = torch.ones((32, 2), device="cuda"), torch.ones((1, 2), device="cuda")
    f32 = torch.empty((32, 32), device="cuda")
    bad = [dict(sa=s[:16]), dict(sa=s[:, :1]), dict(sb=s[:5]), dict(sb=s1[:, :1]), dict(sa=s.double()), dict(sa=s.cpu()),
           dict(b=a[:, :128]), dict(a=a.view(torch.int8)), dict(a=a.t()), dict(a=a[0]), dict(b=a.cpu()),
           dict(out=f32[:16]), dict(out=f32.t()), dict(out=f32.double()), dict(out=f32, out_dtype=torch.bfloat16),
           dict(out_dtype=torch.int32), dict(accumulate=True), dict(out=f32.bfloat16(), accumulate=True),
           dict(a=a[:1].expand(32, 256))]
    for kw in bad:
        args = dict(a=a, sa=s, b=a, sb=s1)
        args.update(kw)
        with pytest.raises(ValueError):
            binding.run_fp8(**args)
    with pytest.raises(ValueError):
        binding.run_fp8(a, s, a, s1, tile="1x1")
    with pytest.raises(binding.GemmError):
        binding.run_fp8(a, s, a, s1, out_dtype=torch.float32, tile="256x256")
    assert binding.run_fp8(a, s, a, s1, out=f32).data_ptr() == f32.data_ptr()
