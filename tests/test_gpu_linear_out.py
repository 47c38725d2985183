"""Results written between the rows of what a call reads: taken where no byte is
shared, whatever the rows' distances; refused where one is."""
import pytest
import torch

from software_pipelined_tiled_02_amd import binding

pytestmark = pytest.mark.gpu


def rand(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


STEPS = (64, 128, 255, 256, 257, 384, 512, 4096)


def test_rows_of_two_distances():
    """32 rows of 64 values, those read 256 apart, in one buffer with those written."""
    buf, w, r = rand(32 * 4096 // 256, 256), rand(64, 64, seed=1), rand(32, 64, seed=2)
    flat = buf.flatten()
    a = buf[:32, :64]
    keep, want = a.clone(), binding.linear(a, w, residual=r)
    places = lambda step, first: {first + step * i + c for i in range(32) for c in range(64)}  # noqa: E731
    read, taken = places(256, 0), 0
    for step in STEPS:
        for first in (0, 63, 64, 65, 128, 190, 192, 193, 250, 8000, 8127):
            if max(written := places(step, first)) >= flat.numel():
                continue
            out = flat[first:].as_strided((32, 64), (step, 1))
            if read & written:
                with pytest.raises(ValueError):
                    binding.linear(a, w, residual=r, out=out)
            else:
                assert binding.linear(a, w, residual=r, out=out) is out
                assert torch.equal(out, want) and torch.equal(a, keep), (step, first)
                taken += 1
    assert taken > 20


def test_one_row_in_a_gap():
    buf, w = rand(16, 256, seed=3), rand(64, 64, seed=4)
    a, one = buf[:, :64], rand(1, 64, seed=5)
    want = binding.linear(one, w, residual=one)
    out = buf[3:4, 64:128]
    assert torch.equal(binding.linear(one, w, residual=one, out=out), want)
    gate = binding.gated(a, w, w)
    assert torch.equal(binding.gated(a, w, w, gate_bias=torch.zeros(64, device="cuda").bfloat16(), out=buf[:, 190:254]), gate)
    bias = buf[5, 64:128]                                          # a bias between the rows of a result
    assert binding.linear(rand(16, 64, seed=6), w, bias=bias, out=buf[:, 128:192]).shape == (16, 64)
    assert binding.linear(rand(16, 64, seed=6), w, bias=bias, out=a) is a
    with pytest.raises(ValueError):
        binding.linear(rand(16, 64, seed=6), w, bias=bias, out=buf[:, 127:191])
    # a weight's gradient in every second column block of a buffer, its bias's beside it
    dc, x = rand(40, 8, seed=7), rand(40, 64, seed=8)
    floats = torch.zeros((8, 128), device="cuda")
    dw, db = binding.weight_gradient(dc, x, bias=True)
    got, sums = binding.weight_gradient(dc, x, out=floats[:, :64], bias_out=floats[2, 64:72])
    assert torch.equal(got, dw) and torch.equal(sums, db)
    with pytest.raises(ValueError):
        binding.weight_gradient(dc, x, out=floats[:, :64], bias_out=floats[2, 63:71])
