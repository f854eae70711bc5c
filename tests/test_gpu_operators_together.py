"""The norm, the products, the update and the answer of a quantized linear
layer, one after the other as a training step and a decoding step use them."""
import pytest
import torch

import mxfp4_block_quantization_quantizer_b200 as m

pytestmark = pytest.mark.gpu


def randn(*shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda")


def test_training_step_then_an_answer():
    rows, k, n = 256, 512, 384
    x = randn(rows, k, seed=1).to(torch.bfloat16)
    gain, off = 1 + 0.1 * randn(k, seed=2), 0.1 * randn(k, seed=3)
    w = 0.02 * randn(n, k, seed=4)                   # fp32 master weight

    # forward: norm and Q_D in one pass, the product of 4-bit operands
    xc, xs, y, mean, rstd = m.layernorm_quantize(x, gain, off, want_y=True, want_stats=True)
    wc, ws = m.quantize(w)
    wb = m.scales_to_blocked(ws)
    out = m.gemm(xc, m.scales_to_blocked(xs), wc, wb, k)
    qy = m.dequantize(xc, xs, rows, k, out_dtype=torch.float32).double()
    qw = m.dequantize(wc, ws, n, k, out_dtype=torch.float32).double()
    bound = (k - 1) * 2.0 ** -24 * (qy.abs() @ qw.abs().T)
    assert ((out.double() - qy @ qw.T).abs() <= bound).all()
    # the same product with y left in bf16
    fine = m.gemv(y, wc, wb, out_dtype=torch.float32)
    bound = (k + 64) * 2.0 ** -24 * 1.25 * (y.double().abs() @ qw.abs().T) + 1e-6
    assert ((fine.double() - y.double() @ qw.T).abs() <= bound).all()

    # backward through the norm, for a gradient that comes from the product
    dout = randn(rows, n, seed=5)
    dy = (dout.double() @ qw).to(torch.bfloat16)
    dx, dgain, doff = m.layernorm_backward(dy, x, mean, rstd, gain)
    xd = x.double().requires_grad_()
    gd, od = gain.double().requires_grad_(), off.double().requires_grad_()
    torch.nn.functional.layer_norm(xd, (k,), gd, od, 1e-5).backward(dy.double())
    for got, want, eps in ((dx, xd.grad, 2.0 ** -8), (dgain, gd.grad, 2.0 ** -18),
                           (doff, od.grad, 2.0 ** -18)):
        assert (got.double() - want).norm() <= eps * want.norm()

    # update: the weight's gradient made orthogonal, Q-Ramping, Q-EMA
    grad = (dout.double().T @ y.double()).float()
    delta = m.newton_schulz(grad, scale=-0.01)
    sv = torch.linalg.svdvals(delta.double()) / 0.01
    # (256 rows: a gradient of rank 256, whose values five steps bring near 1)
    assert sv.max() < 1.3 and sv[:192].min() > 0.6 and sv[256:].max() < 0.05
    w0, zeros = w.clone(), [torch.zeros_like(w) for _ in range(4)]
    m.qramp_step(w, delta, *zeros, torch.zeros(w.shape, dtype=torch.uint8, device="cuda"), 0)
    assert torch.equal(w, w0 + delta)
    ema = w0.clone()
    ec, es = m.qema_quantize(w, ema, 0.998)

    # answer: one token, a batch of tokens and a graph of both, on the averaged weight
    eb = m.scales_to_blocked(es)
    ew = m.dequantize(ec, es, n, k, out_dtype=torch.float32).double()
    tokens = randn(5, k, seed=6).to(torch.bfloat16)

    def answer():
        h = m.layernorm(tokens, gain, off)
        return m.gemv(h, ec, eb), m.gemv(h[:1], ec, eb)
    batch, one = answer()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gb, go = answer()
    for seed in (7, 8):
        tokens.copy_(randn(5, k, seed=seed))
        graph.replay()
        batch, one = answer()
        assert torch.equal(gb, batch) and torch.equal(go, one)
        want = m.layernorm(tokens, gain, off).double() @ ew.T
        assert (batch.double() - want).norm() <= 2.0 ** -8 * want.norm()
        assert (one.double() - want[:1]).norm() <= 2.0 ** -8 * want[:1].norm()


def test_two_graphs_and_eager_calls_share_nothing():
    """Two captured graphs of the operators with workspaces, replayed one over
    the other on two streams while eager calls run on a third."""
    codes, scales = m.quantize(0.02 * randn(1024, 1024, seed=10))
    blocked = m.scales_to_blocked(scales)
    gain = 1 + 0.1 * randn(1024, seed=11)
    xs = [randn(40, 1024, seed=s).to(torch.bfloat16) for s in (12, 13, 14)]

    def work(x):
        y, mean, rstd = m.layernorm(x, gain, want_stats=True)
        z = m.gemv(y, codes, blocked)
        return (z, *m.layernorm_backward(z, x, mean, rstd, gain), m.newton_schulz(z))
    want = [[t.clone() for t in work(x)] for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    graphs, outs = [], []
    for x, s in zip(xs[:2], streams):
        g = torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            outs.append(work(x))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = work(xs[2])
    torch.cuda.synchronize()
    for got, ref in zip(outs + [eager], want):
        for a, b in zip(got, ref):
            assert torch.equal(a, b)


def test_side_stream_owns_its_memory():
    """Work queued on a side stream keeps its workspace and outputs while the
    current stream goes on allocating and writing."""
    codes, scales = m.quantize(0.02 * randn(1024, 1024, seed=20))
    blocked = m.scales_to_blocked(scales)
    gain = 1 + 0.1 * randn(1024, seed=21)
    x = randn(40, 1024, seed=22).to(torch.bfloat16)
    dy = randn(40, 1024, seed=23).to(torch.bfloat16)

    def work(stream=None):
        y, mean, rstd = m.layernorm(x, gain, want_stats=True, stream=stream)
        q = m.layernorm_quantize(x, gain, stream=stream)
        z = m.gemv(x, codes, blocked, stream=stream)
        return (y, mean, rstd, *q, z,
                *m.layernorm_backward(dy, x, mean, rstd, gain, stream=stream),
                m.newton_schulz(x, stream=stream))
    want = work()
    side = torch.cuda.Stream()
    sizes = [t.numel() * t.element_size() for t in want]
    sizes += [1 << b for b in range(9, 22)]
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)     # the side stream starts late
        got = work(side)
        junk = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del got, junk


def test_layernorm_past_32_bit_offsets():
    """More than 2^31 elements: the last rows are those of a call on them
    alone, and the first ones too (a row's bits depend on its content and the
    split of a row over warps, which follows from the columns)."""
    cols, rows = 2048, (1 << 20) + 77
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x.view(-1)[:] = 1.0
    ends = randn(2 * 2048, cols, seed=30).to(torch.bfloat16)
    x[:2048], x[-2048:] = ends[:2048], ends[2048:]
    w, b = 1 + 0.1 * randn(cols, seed=31), randn(cols, seed=32)
    y, mean, rstd = m.layernorm(x, w, b, want_stats=True)
    codes, scales = m.layernorm_quantize(x, w, b)
    assert torch.equal(y[5000], b.to(torch.bfloat16))           # a constant row
    small = m.layernorm(ends, w, b, want_stats=True)
    qc, qs = m.layernorm_quantize(ends, w, b)
    for got, want in zip((y, mean, rstd, codes, scales), (*small, qc, qs)):
        assert torch.equal(got[:2048], want[:2048])
        assert torch.equal(got[-2048:], want[2048:])
    dx, dw, db = m.layernorm_backward(x, x, mean, rstd, w)
    sx, _, _ = m.layernorm_backward(ends, ends, *small[1:], w)
    assert torch.equal(dx[:2048], sx[:2048]) and torch.equal(dx[-2048:], sx[2048:])
    # constant rows have h = 0: dw is that of the ends; db counts every row
    h = (ends.double() - small[1].double()[:, None]) * small[2].double()[:, None]
    want_w = (ends.double() * h).sum(0)
    # each product is off by 2^-22 of its size, the fixed-order fp32 sums by
    # at most 2^-24 for each of the (rows / CTA + CTAs) additions that are not
    # of zeros: 4096 bounds them
    tol = (2.0 ** -22 + 4096 * 2.0 ** -24) * (ends.double() * h).abs().sum(0) + 1e-6
    assert ((dw.double() - want_w).abs() <= tol).all()
    want_b = ends.double().sum(0) + (rows - 4096)
    # about 2^20 ones: sums of a CTA (below 2^24) are off by 2^-24 of what
    # they hold at each of about 7200 additions
    tol = 8192 * 2.0 ** -24 * (ends.double().abs().sum(0) + (rows - 4096))
    assert ((db.double() - want_b).abs() <= tol).all()


@pytest.mark.parametrize("rows", [1, 3, 17])
def test_gemv_past_32_bit_offsets(rows):
    """A weight of more than 2^31 bytes of codes: its last row block."""
    n, k = 65536 + 64, 65536
    g = torch.Generator(device="cuda")
    g.manual_seed(33)
    codes = torch.zeros(n, k // 2, dtype=torch.uint8, device="cuda")
    last = n - n % 128 - 128
    codes[last:] = torch.randint(0, 256, (n - last, k // 2), dtype=torch.uint8, device="cuda",
                                 generator=g)
    scales = torch.full((n, k // 32), 120, dtype=torch.uint8, device="cuda")
    blocked = m.scales_to_blocked(scales)
    x = randn(rows, k, seed=34).to(torch.bfloat16)
    y = m.gemv(x, codes, blocked, out_dtype=torch.float32)
    assert (y[:, :last] == 0).all()
    w = m.dequantize(codes[last:].contiguous(), scales[last:].contiguous(), n - last, k,
                     out_dtype=torch.float32).double()
    want = x.double() @ w.T
    bound = (k + 64) * 2.0 ** -24 * 1.25 * (x.double().abs() @ w.abs().T) + 1e-6
    assert ((y[:, last:].double() - want).abs() <= bound).all()


FIRST_CALLS = """
import torch
import mxfp4_block_quantization_quantizer_b200 as m
g = torch.Generator(device="cuda")
g.manual_seed(40)
new = lambda *s: torch.randn(s, generator=g, device="cuda")
x, dy, wide = new(700, 1024).bfloat16(), new(700, 1024).bfloat16(), new(20, 14336)
codes = torch.randint(0, 256, (256, 512), generator=g, device="cuda", dtype=torch.uint8)
blocked = torch.full((256, 32), 120, dtype=torch.uint8, device="cuda")

def work():
    out = []
    for t, d in ((x, dy), (wide, wide)):
        y, mean, rstd = m.layernorm(t, want_stats=True)
        out += [y, mean, rstd, *m.layernorm_backward(d, t, mean, rstd)]
        out += list(m.layernorm_quantize(t))
    out += [m.gemv(x[:n], codes, blocked) for n in (1, 5, 12, 40)]
    return out + [m.newton_schulz(t) for t in (x, wide)]

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = work()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
for a, b in zip(got, work()):
    assert torch.equal(a, b)
print("same")
"""


def test_first_calls_of_a_process_are_captured():
    """No call before the capture has loaded a kernel or set its limits."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True,
                          text=True, timeout=300)
    assert done.returncode == 0 and "same" in done.stdout, done.stderr[-2000:]
