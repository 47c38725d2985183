"""The feed-forward operators one after another, as a block's training step and
a decoding step use them: every result against its definition in 64 bits, on
streams, in threads and captured in graphs."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from software_pipelined_tiled_02_amd import binding
from tests import linear_ref as R
from tests.linear_ref import FT, assert_within

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def block(M, D, F, dtype="bf16", seed=0):
    """x, gate, up, down, gate's bias, and the gradient of the block's output."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s, size=1.0: (size * torch.randn(s, generator=g, device="cuda")).to(FT[dtype])  # noqa: E731
    return [n(M, D), n(F, D, size=D ** -0.5), n(F, D, size=D ** -0.5), n(D, F, size=F ** -0.5), n(F), n(M, D)]


def step(x, wg, wu, wd, bg, dy, grads=None, activation="silu"):
    """y = x + (act(x wg^T + bg) * (x wu^T)) wd^T and its gradients; the weights' are added to `grads` where given."""
    h, g, u = binding.gated(x, wg, wu, gate_bias=bg, activation=activation, keep=True)
    y = binding.linear(h, wd, residual=x)
    dg, du, again = binding.gated_backward(dy, wd, g, u, activation=activation, keep=True)
    dx = binding.linear(dg, wg, layout="RR", pair=(du, wu), residual=dy)
    add = (lambda i: {}) if grads is None else lambda i: dict(out=grads[i], accumulate=True)
    dwg, dbg = binding.weight_gradient(dg, x, bias=True, **add(0), **({} if grads is None else dict(bias_out=grads[3])))
    dwu = binding.weight_gradient(du, x, **add(1))
    dwd = binding.weight_gradient(dy, again, **add(2))
    return dict(h=h, g=g, u=u, y=y, dg=dg, du=du, again=again, dx=dx, dwg=dwg, dbg=dbg, dwu=dwu, dwd=dwd)


@pytest.mark.parametrize("dtype", ("bf16", "f16"))
@pytest.mark.parametrize("M,D,F,activation", ((1, 64, 192, "silu"), (70, 136, 200, "gelu"), (333, 513, 257, "gelu_tanh"),
                                              (1000, 320, 1112, "silu"), (5, 1026, 66, "relu")))
def test_training_step(M, D, F, activation, dtype):
    x, wg, wu, wd, bg, dy = args = block(M, D, F, dtype)
    o = step(*args, activation=activation)
    d = {k: v.double() for k, v in o.items()}
    x, wg, wu, wd, bg, dy = (t.double() for t in args)
    # each from what the operator was given
    for name, (want, off) in zip("hgu", R.gated(x, wg, wu, dtype, activation, bg)):
        assert_within(o[name], want, off, name)
    assert_within(o["y"], *R.linear(d["h"], wd.t(), dtype, residual=x)[:2], "y")
    for name, (want, off) in zip(("dg", "du", "again"), R.gated_backward(dy, wd, d["g"], d["u"], dtype, activation)):
        assert_within(o[name], want, off, name)
    assert_within(o["dx"], *R.linear(d["dg"], wg, dtype, residual=dy, pair=(d["du"], wu))[:2], "dx")
    for names, dc, a in ((("dwg", "dbg"), d["dg"], x), (("dwu",), d["du"], x), (("dwd",), dy, d["again"])):
        dw, off, db, db_off = R.weight_gradient(dc, a)
        assert_within(o[names[0]], dw, off, names[0])
        if len(names) == 2:
            assert_within(o[names[1]], db, db_off, names[1])


def test_gradients_against_differences():
    """A weight is moved along its gradient: what the loss changes by in 64 bits
    is the gradient's square.  A gradient stands behind at most three roundings in
    a row (g or u, dg or du, the last), each by 2^-8 of a value at most and not
    all one way: less than 2^-6 of its norm."""
    x, wg, wu, wd, bg, dy = args = block(96, 128, 160, "bf16", 3)
    o = step(*args)
    f = [t.double() for t in (x, wg, wu, wd, bg)]

    def loss(x, wg, wu, wd, bg):
        return float(((R.act(x @ wg.t() + bg, "silu") * (x @ wu.t()) @ wd.t() + x) * dy.double()).sum())

    for i, name in enumerate(("dx", "dwg", "dwu", "dwd", "dbg")):
        grad = o[name].double()
        move = 1e-5 / float(grad.norm())
        up, down = (loss(*f[:i], f[i] + s * move * grad, *f[i + 1:]) for s in (1, -1))
        want = float(grad.square().sum())
        assert abs((up - down) / (2 * move) - want) < 2.0 ** -6 * want, name


def test_two_batches_add_up():
    """Gradients of two batches added in place: the first one's bits, and one addition more."""
    one, two = block(130, 200, 264, seed=1), block(130, 200, 264, seed=2)
    two[1:5] = one[1:5]
    grads = [torch.zeros(s, device="cuda") for s in ((264, 200), (264, 200), (200, 264), (264,))]
    a, b = step(*one), step(*two)
    step(*one, grads=grads)
    step(*two, grads=grads)
    for got, name in zip(grads, ("dwg", "dwu", "dwd", "dbg")):
        assert torch.equal(got, b[name] + a[name]), name


def test_decoding_one_token_is_a_row_of_the_batch():
    """Rows are independent: each token by itself, against its definition."""
    x, wg, wu, wd, bg, _ = block(9, 320, 456, seed=4)
    for i in range(9):
        row = x[i:i + 1]
        h = binding.gated(row, wg, wu, gate_bias=bg)
        y = binding.linear(h, wd, residual=row)
        assert_within(h, *R.gated(row.double(), wg.double(), wu.double(), "bf16", "silu", bg.double())[0], "h")
        assert_within(y, *R.linear(h.double(), wd.double().t(), "bf16", residual=row.double())[:2], "y")


SIZES = ((1, 512, 640), (70, 400, 272), (700, 520, 1100))


@pytest.mark.parametrize("M,D,F", SIZES)
def test_captured_and_replayed(M, D, F):
    """Two graphs of the step in one pool, replayed in turn between eager steps that allocate."""
    static = block(M, D, F)
    grads = [torch.zeros(s, device="cuda") for s in ((F, D), (F, D), (D, F), (F,))]
    step(*static, grads=grads)
    torch.cuda.synchronize()
    graphs, pool = [], None
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            out = step(*static, grads=grads)
        pool = g.pool()
        graphs.append((g, out))
    for seed in range(1, 5):
        for t, v in zip(static, block(M, D, F, seed=seed)):
            t.copy_(v)
        for g, out in graphs:
            want = [torch.zeros_like(t) for t in grads]
            eager = step(*static, grads=want)
            for t in grads:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(grads, want))
            for name in eager:
                assert torch.equal(out[name], eager[name]), name


def test_streams_and_raw_handles():
    """On a stream of its own, behind that stream's work, by torch's object and its raw handle."""
    args = block(200, 264, 392, seed=5)
    want = step(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for how in ("current", "object", "raw"):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            x = torch.zeros_like(args[0])
            for _ in range(30):
                x += 0.25                                  # work ahead on the stream, whose result the operators need
            x.copy_(args[0])
        stream = side if how == "object" else side.cuda_stream
        if how == "current":
            with torch.cuda.stream(side):
                got = step(x, *args[1:])
        else:
            h, g, u = binding.gated(x, args[1], args[2], gate_bias=args[4], keep=True, stream=stream)
            y = binding.linear(h, args[3], residual=x, stream=stream)
            dg, du = binding.gated_backward(args[5], args[3], g, u, stream=stream)
            got = dict(h=h, g=g, u=u, y=y, dg=dg, du=du, dwu=binding.weight_gradient(du, x, stream=stream))
        side.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in got), how


def test_threads_at_once():
    args = [block(150, 200, 328, seed=i) for i in range(4)]
    want = [step(*a) for a in args]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got = step(*args[i])
                    stream.synchronize()
                    if not all(torch.equal(got[k], want[i][k]) for k in got):
                        wrong.append(i)
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


FIRST_CALL = """
import torch
from software_pipelined_tiled_02_amd import binding
x, w = (torch.ones((n, 64), device="cuda").bfloat16() for n in (4, 32))
z = torch.ones((4, 32), device="cuda").bfloat16()
torch.cuda.synchronize()
calls = (lambda: binding.linear(x, w), lambda: binding.gated(x, w, w), lambda: binding.gated_backward(x, w.t().contiguous(), z),
         lambda: binding.weight_gradient(z, x))
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for call in calls:
        try:
            call()
            raise SystemExit("not refused")
        except RuntimeError as e:
            assert "before the graph capture" in str(e), e
    y = x + 1
g.replay()
c = binding.linear(y, w)
torch.cuda.synchronize()
assert bool((c == 128).all())
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):                      # one eager call is enough for the others
    h = binding.gated(x, w, w, activation="none")
    dw = binding.weight_gradient(h, x)
for i in range(3):
    x.fill_(i + 1)
    g.replay()
    torch.cuda.synchronize()
    assert bool((h == (64 * (i + 1)) ** 2).all()) and bool((dw == 4 * (64 * (i + 1)) ** 2 * (i + 1)).all())
print("refused, then fine")
"""


def test_first_call_under_capture_is_refused():
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=ROOT, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "refused, then fine" in r.stdout, r.stdout + r.stderr
