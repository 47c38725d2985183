"""What the 8-bit operators write in place is noticed by torch's autograd."""
import pytest
import torch

from software_pipelined_tiled_02_amd import binding

pytestmark = pytest.mark.gpu


def rand(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def test_what_is_written_in_place_is_noticed():
    x, w = rand(6, 256), rand(256, seed=1)
    q, s = binding.quantize_fp8(x)
    h, rstd = binding.rms_fp8(x, w)[2:4]
    for call, kept in ((lambda t: binding.run_fp8(q, s, q, s, out=t), torch.zeros((6, 6), device="cuda")),
                       (lambda t: binding.rms_fp8(x, w, residual=t, h_out=t), rand(6, 256, seed=2)),
                       (lambda t: binding.rms_backward(t, h, w, rstd, dx_out=t), rand(6, 256, seed=3))):
        a = torch.ones((), device="cuda", requires_grad=True)
        y = a * kept                                              # keeps `kept`
        call(kept)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
    with torch.inference_mode():                                  # such tensors count no versions
        t = torch.zeros((6, 6), device="cuda")
    assert binding.run_fp8(q, s, q, s, out=t) is t
