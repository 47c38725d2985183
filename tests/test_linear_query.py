"""gemm_query_linear names the kernel that a call with a second product takes,
where that is another one than the single product's (no GPU)."""
import pytest

from software_pipelined_tiled_02_amd import binding

SIZES = [(M, N, K) for M in (1, 16, 64, 130, 1000) for N in (64, 512, 4096) for K in (1, 64, 200, 4096)]


def q(form, M, N, K, **kw):
    rc, info = binding.gemm_query_linear(form, M, N, K, **kw)
    assert rc == binding.GEMM_OK
    return info


def test_a_second_product_counts():
    """Twice the K-tiles in the choice: the class of a single product over 2 K, in whole K-tiles."""
    differ = 0
    for layout in ("rc", "rr"):
        for M, N, K in SIZES:
            for r16 in (True, False):
                one, two = (q("linear_%s%s" % (layout, pair), M, N, K, rows16=r16) for pair in ("", "_pair"))
                same = q("linear_" + layout, M, N, 2 * (-(-K // 64)) * 64, rows16=r16)
                assert two["tile"] == same["tile"] and two["grid"] == same["grid"], (layout, M, N, K, r16)
                assert two["k_tiles"] == one["k_tiles"] == -(-K // 64)
                differ += one["tile"] != two["tile"]
    assert differ > 0


def test_the_size_where_it_was_seen():
    info = q("linear_rr_pair", 1, 4096, 64)
    assert info["tile"] == binding.LINEAR_TILES["16x16"] and q("linear_rr", 1, 4096, 64)["tile"] != info["tile"]


@pytest.mark.parametrize("form", ("linear_rc_pair", "linear_rr_pair"))
def test_every_class_is_there(form):
    for tile, number in binding.LINEAR_TILES.items():
        if tile != "auto":
            assert q(form, 300, 300, 100, tile=tile)["tile"] == number


def test_other_numbers_are_refused():
    for form in [n for n in range(-40, 40) if n not in binding.LINEAR_FORMS.values()]:
        assert binding.gemm_query_linear(form, 1, 1, 1, check=False)[0] == binding.GEMM_ERR_INVALID_ARG, form
