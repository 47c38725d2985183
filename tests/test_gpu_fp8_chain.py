"""One linear layer through 8 bits, forward and backward, as a training step
and a decoding step use it: every stage against its definition on what the
stage before it gave, the whole against unquantised arithmetic, and the same
captured in a graph and replayed."""
import subprocess
import sys

import numpy as np
import pytest
import torch

from software_pipelined_tiled_02_amd import binding
from tests import fp8_ref as R
from tests.conftest import ROOT
from tests.fp8_util import check_product, raw_of

pytestmark = pytest.mark.gpu


def layer(M, D, N, seed):
    g = torch.Generator().manual_seed(seed)
    x, r = (torch.randn((M, D), generator=g).bfloat16() for _ in range(2))
    wn = (1 + 0.2 * torch.randn((D,), generator=g)).bfloat16()
    w = 0.05 * torch.randn((N, D), generator=g)
    dc, dh = torch.randn((M, N), generator=g).bfloat16(), torch.randn((M, D), generator=g).bfloat16()
    return [t.cuda() for t in (x, r, wn, w, dc, dh)]


def step(x, r, wn, w, dc, dh, grad):
    """c = norm(x + r) w^T forward; gradients of x (and r), wn, and w (added to grad)."""
    wq, ws, wqt, wst = binding.quantize_fp8(w, block="tile", transpose=True)
    q, s, h, rstd, y = binding.rms_fp8(x, wn, residual=r, norm=True)
    c = binding.run_fp8(q, s, wq, ws)
    dq, ds, dqt, dst = binding.quantize_fp8(dc, transpose=True)
    dy = binding.run_fp8(dq, ds, wqt, wst)
    yqt, yst = binding.quantize_fp8(y, rows=False, transpose=True)
    binding.run_fp8(dqt, dst, yqt, yst, out=grad, accumulate=True)
    dx, dwn = binding.rms_backward(dy, h, wn, rstd, dh=dh)
    return dict(c=c, dx=dx, dwn=dwn, dy=dy, q=q, s=s, h=h, rstd=rstd, y=y, wq=wq, ws=ws, wqt=wqt, wst=wst, dq=dq, ds=ds,
                dqt=dqt, dst=dst, yqt=yqt, yst=yst)


@pytest.mark.parametrize("M,D,N", ((37, 272, 200), (130, 128, 144), (1, 300, 40)))
def test_training_step(M, D, N):
    args = layer(M, D, N, 3)
    x, r, wn, w, dc, dh = args
    grad = torch.ones((N, D), device="cuda")
    o = step(*args, grad)
    f = lambda n: o[n].cpu().numpy()  # noqa: E731
    check_product(o["c"], raw_of(o["q"]), f("s"), raw_of(o["wq"]), f("ws"), "e4m3", "e4m3", 128, "bf16", "c")
    check_product(o["dy"], raw_of(o["dq"]), f("ds"), raw_of(o["wqt"]), f("wst"), "e4m3", "e4m3", 128, "bf16", "dy")
    check_product(grad, raw_of(o["dqt"]), f("dst"), raw_of(o["yqt"]), f("yst"), "e4m3", "e4m3", 1, "f32", "dw",
                  base=np.ones((N, D)))
    assert np.array_equal(raw_of(o["wqt"]), raw_of(o["wq"]).T) and torch.equal(o["wst"], o["ws"].t())
    # the whole step without 8 bits: every product's factors are off by 2^-4 at
    # most, each (independent, so over 2^-5 of the 2-norm for sums of many)
    h = (x.float() + r.float()).bfloat16().double()
    y = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * wn.double()
    c = y @ w.double().t()
    dy = dc.double() @ w.double()
    dw = dc.double().t() @ y
    dx, dwn = R.rms_backward(dy.cpu().numpy(), h.cpu().numpy(), wn.double().cpu().numpy(),
                             (h.square().mean(1) + 1e-6).rsqrt().cpu().numpy(), dh.double().cpu().numpy())
    for got, ref in ((o["c"], c), (o["dy"], dy), (grad - 1, dw), (o["dx"], torch.from_numpy(dx)),
                     (o["dwn"], torch.from_numpy(dwn))):
        got, ref = got.double().cpu(), ref.cpu()
        assert float((got - ref).norm() / ref.norm()) < 2 * 2.0 ** -4


def test_training_step_captured_and_replayed():
    M, D, N = 70, 400, 272
    static = layer(M, D, N, 0)
    grad = torch.zeros((N, D), device="cuda")
    step(*static, grad)                                            # eager once: handles, library
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):                                             # two graphs of the same step
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(*static, grad)
        graphs.append((g, out))
    for seed in range(1, 5):
        for t, v in zip(static, layer(M, D, N, seed)):
            t.copy_(v)
        eager_grad = torch.zeros((N, D), device="cuda")
        eager = step(*static, eager_grad)
        torch.cuda.synchronize()
        for g, out in graphs:
            grad.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(grad, eager_grad)
            for name in ("c", "dx", "dwn", "q", "s"):
                assert torch.equal(out[name].view(torch.uint8) if name == "q" else out[name],
                                   eager[name].view(torch.uint8) if name == "q" else eager[name]), name


FIRST_CALL = """
import torch
from software_pipelined_tiled_02_amd import binding
x = torch.ones((4, 256), device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    try:
        binding.quantize_fp8(x)
        raise SystemExit("not refused")
    except RuntimeError as e:
        assert "before the graph capture" in str(e), e
    y = x + 1
g.replay()
q, s = binding.quantize_fp8(y)
torch.cuda.synchronize()
assert bool((q.float() * s.repeat_interleave(128, 1) == 2).all())
print("refused, then fine")
"""


def test_first_call_under_capture_is_refused():
    """A process's first call on a device sets it up, which a capture cannot
    hold: an error, and neither a broken graph nor a broken process."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=ROOT, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "refused, then fine" in r.stdout, r.stdout + r.stderr


def test_threads_at_once():
    """Calls from several host threads, each on a stream of its own."""
    import threading
    args = layer(64, 256, 128, 1)
    ref = step(*args, torch.zeros((128, 256), device="cuda"))
    torch.cuda.synchronize()
    wrong = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(5):
                o = step(*args, torch.zeros((128, 256), device="cuda"))
                s.synchronize()
                if not (torch.equal(o["c"], ref["c"]) and torch.equal(o["dx"], ref["dx"]) and torch.equal(o["dwn"], ref["dwn"])):
                    wrong.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
