"""Layer norm and its gradients against the formulas in 64 bits.

Tolerances are forward error bounds of the kernels' fp32 arithmetic. With
u = 2^-24: a sum over a row is at most `depth` additions deep (32 elements a
thread, then at most 10 joining steps; wider rows add cols / 512), so it is
off by at most depth u times the sum of magnitudes; every other operation
adds u of its result; an output rounded to its type is off by half a step.
"""
import numpy as np
import pytest
import torch

import mxfp4_block_quantization_quantizer_b200 as m

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F = torch.bfloat16, torch.float32
SHAPES = [(1, 1), (1, 4096), (3, 5), (7, 48), (9, 63), (64, 384), (197, 1536), (700, 256),
          (33, 1111), (620, 1111), (5, 16384), (3, 16392), (2, 20001), (2, 40000), (300, 8192),
          (1300, 96), (1201, 2048), (310, 5000), (12, 9001), (5003, 8), (2999, 640), (4001, 264),
          (901, 4096), (595, 4104), (3333, 1000)]


def depth(cols):
    return 64 + (cols // 512 if cols > 16384 else 0)


def half_step(t):
    return 0.5 * torch.finfo(t).eps


def inputs(rows, cols, dt, seed, offset=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    chan = torch.exp2(6 * torch.rand(cols, generator=g, device="cuda") - 3)
    x = (torch.randn(rows, cols, generator=g, device="cuda") * chan + offset).to(dt)
    dy = torch.randn(rows, cols, generator=g, device="cuda").to(dt)
    w = 1 + 0.3 * torch.randn(cols, generator=g, device="cuda")
    b = 0.2 * torch.randn(cols, generator=g, device="cuda")
    return x, dy, w, b


def forward64(x, w, b, eps):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    var = (x - mean).square().mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    h = (x - mean) * rstd
    y = h if w is None else h * w.double()
    return (y if b is None else y + b.double()), mean, rstd, h


def check_forward(x, w, b, eps, got, mean, rstd):
    y, mu, rs, h = forward64(x, w, b, eps)
    d = depth(x.shape[1])
    aw = 1.0 if w is None else w.double().abs()
    ab = 0.0 if b is None else b.double().abs()
    dm = d * U * x.double().abs().mean(1, keepdim=True)      # of the mean
    dr = d * U + (dm * rs) ** 2                              # of rstd, relative
    tol = aw * (dm * rs + h.abs() * dr) + 4 * U * (y.abs() + ab) + 1e-30
    tol = tol + half_step(x.dtype) * (y.abs() + tol)
    assert ((got.double() - y).abs() <= tol).all(), ((got.double() - y).abs() / tol).max()
    assert ((mean.double() - mu[:, 0]).abs() <= dm[:, 0] + 1e-37).all()
    assert ((rstd.double() - rs[:, 0]).abs() <= dr[:, 0] * rs[:, 0]).all()


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, dt):
    x, _, w, b = inputs(*shape, dt, 1)
    check_forward(x, w, b, 1e-5, *m.layernorm(x, w, b, want_stats=True))


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("use_w,use_b", [(False, False), (True, False), (False, True)])
def test_forward_without_parameters(dt, use_w, use_b):
    x, _, w, b = inputs(40, 768, dt, 2)
    w, b = (w if use_w else None), (b if use_b else None)
    y, mean, rstd = m.layernorm(x, w, b, 1e-6, want_stats=True)
    check_forward(x, w, b, 1e-6, y, mean, rstd)
    assert torch.equal(m.layernorm(x, w, b, 1e-6), y)


@pytest.mark.parametrize("cols", [768, 771, 18000])
def test_forward_with_a_large_offset(cols):
    """A common offset of 1e4 in fp32 data of unit size: the squares are
    summed around the mean, so only x itself has lost bits."""
    x, _, w, b = inputs(50, cols, F, 3, offset=1e4)
    check_forward(x, w, b, 1e-5, *m.layernorm(x, w, b, want_stats=True))


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("cols", [96, 1000, 1003, 17000])
def test_strided_and_unaligned_rows(dt, cols):
    """Views of a wider tensor: class tokens (every third row), and columns
    that start off a 16-byte boundary."""
    x, dy, w, b = inputs(60, 2 * cols + 1, dt, 4)
    for xv, dv in ((x[::3, :cols], dy[1::3, 8:cols + 8]), (x[:, 1:cols + 1], dy[:, :cols])):
        y, mean, rstd = m.layernorm(xv, w[:cols], b[:cols], want_stats=True)
        assert y.is_contiguous()
        check_forward(xv, w[:cols], b[:cols], 1e-5, y, mean, rstd)
        check_backward(dv, xv, mean, rstd, w[:cols],
                       *m.layernorm_backward(dv, xv, mean, rstd, w[:cols].clone()))
    ws = torch.zeros(cols + 1, device="cuda")[1:]     # a weight off a 16-byte boundary
    ws.copy_(w[:cols])
    xc = x[:, :cols].contiguous()
    assert torch.allclose(m.layernorm(xc, ws, b[:cols]).float(),
                          m.layernorm(xc, w[:cols].contiguous(), b[:cols]).float(),
                          rtol=2 * half_step(dt) + 64 * U, atol=1e-5)


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("cols", [512, 515, 17001])
def test_special_rows(dt, cols):
    """A constant row gives the bias; rows with NaN or Inf give NaN and touch
    no other row; magnitudes near the type's ends stay finite."""
    x, _, w, b = inputs(8, cols, dt, 5)
    x[1] = 3.5
    x[2, cols // 2] = float("nan")
    x[3, 1] = float("inf")
    x[4] *= 2.0 ** 50
    x[5] *= 2.0 ** -60
    y, mean, rstd = m.layernorm(x, w, b, want_stats=True)
    assert torch.isnan(y[2]).all() and torch.isnan(y[3]).all()
    keep = [0, 1, 4, 5, 6, 7]
    check_forward(x[keep], w, b, 1e-5, y[keep], mean[keep], rstd[keep])


def check_backward(dy, x, mean, rstd, w, dx, dw=None, db=None):
    rows, cols = x.shape
    dyd, rs = dy.double(), rstd.double()[:, None]
    h = (x.double() - mean.double()[:, None]) * rs
    g = dyd if w is None else dyd * w.double()
    c1, c2 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    want = rs * (g - c1 - h * c2)
    d = depth(cols)
    tol = rs.abs() * (4 * U * g.abs() + d * U * g.abs().mean(1, keepdim=True)
                      + h.abs() * ((d + 4) * U * (g * h).abs().mean(1, keepdim=True)
                                   + 4 * U * c2.abs())) + 4 * U * want.abs() + 1e-30
    tol = tol + half_step(x.dtype) * (want.abs() + tol)
    assert ((dx.double() - want).abs() <= tol).all(), ((dx.double() - want).abs() / tol).max()
    if dw is not None:
        # at most rows / 148 rows in one chain (fewer CTAs only where there
        # are fewer rows; 64 chains for wide rows), then the partial rows
        r = rows / 64 + 64
        for got, terms in ((dw, dyd * h), (db, dyd)):
            bound = (r + 4) * U * terms.abs().sum(0) + 1e-30
            assert ((got.double() - terms.sum(0)).abs() <= bound).all()


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, dt):
    x, dy, w, _ = inputs(*shape, dt, 6)
    _, mean, rstd = m.layernorm(x, w, want_stats=True)
    out = m.layernorm_backward(dy, x, mean, rstd, w)
    check_backward(dy, x, mean, rstd, w, *out)
    dx = m.layernorm_backward(dy, x, mean, rstd, w, want_params=False)
    check_backward(dy, x, mean, rstd, w, dx)
    for a, b in zip(out, m.layernorm_backward(dy, x, mean, rstd, w)):
        assert torch.equal(a, b)      # no order left to chance


@pytest.mark.parametrize("dt", [BF, F])
def test_backward_without_weight(dt):
    x, dy, _, _ = inputs(77, 640, dt, 7)
    _, mean, rstd = m.layernorm(x, want_stats=True)
    check_backward(dy, x, mean, rstd, None, *m.layernorm_backward(dy, x, mean, rstd))


def test_backward_against_differences():
    """Directional derivative of sum(c y) against a central difference of the
    formula in 64 bits: step s gives an error of order s^2."""
    x, c, w, b = inputs(6, 40, F, 8)
    _, mean, rstd = m.layernorm(x, w, b, want_stats=True)
    dx, dw, db = (t.double() for t in m.layernorm_backward(c, x, mean, rstd, w))
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    vx, vw, vb = (torch.randn(t.shape, generator=g, device="cuda").double() for t in (x, w, b))
    s = 1e-5
    f = lambda k: (c.double() * forward64(x.double() + k * vx, w.double() + k * vw,
                                          b.double() + k * vb, 1e-5)[0]).sum()
    want = (f(s) - f(-s)) / (2 * s)
    got = (dx * vx).sum() + (dw * vw).sum() + (db * vb).sum()
    # fp32 gradients: each is off by a few hundred u of its terms' magnitudes
    bound = 512 * U * ((dx * vx).abs().sum() + (dw * vw).abs().sum() + (db * vb).abs().sum())
    assert (got - want).abs() <= bound + 1e-4 * s * want.abs()


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("shape", [(1, 32), (5, 96), (64, 384), (197, 1536), (400, 1024),
                                   (6, 16384), (3, 16416), (2, 32768), (600, 4096)])
def test_quantize_is_the_quantizer_of_the_norm(shape, dt):
    x, _, w, b = inputs(*shape, dt, 10)
    if shape[0] > 4:
        x[1] = 0
        x[2, 3] = float("nan")
        x[3] *= 2.0 ** 40
    y, mean, rstd = m.layernorm(x, w, b, want_stats=True)
    codes, scales = m.quantize(y)
    got = m.layernorm_quantize(x, w, b, want_y=True, want_stats=True)
    same = lambda a, c: torch.equal(a.view(torch.uint8), c.view(torch.uint8))
    assert torch.equal(got[0], codes) and torch.equal(got[1], scales)
    assert same(torch.nan_to_num(got[2]), torch.nan_to_num(y))
    assert same(torch.nan_to_num(got[3]), torch.nan_to_num(mean))
    alone = m.layernorm_quantize(x, w, b)
    assert torch.equal(alone[0], codes) and torch.equal(alone[1], scales)


def test_outputs_end_where_they_should():
    """Bytes on both sides of every output stay as they were."""
    for rows, cols, dt in ((5, 1111, BF), (9, 4096, F), (3, 20001, F), (700, 40, BF)):
        x, dy, w, b = inputs(rows, cols, dt, 11)
        n = rows * cols
        bufs = [torch.full((64 + k + 64,), 7.0, dtype=t, device="cuda")
                for k, t in ((n, dt), (rows, F), (rows, F), (n, dt), (cols, F), (cols, F))]
        y, mean, rstd, dx, dw, db = (t[64:-64] for t in bufs)
        m.layernorm(x, w, b, want_stats=True, out=(y.view(rows, cols), mean, rstd))
        m.layernorm_backward(dy, x, mean, rstd, w, out=(dx.view(rows, cols), dw, db))
        torch.cuda.synchronize()
        for t in bufs:
            assert (t[:64] == 7).all() and (t[-64:] == 7).all()


def test_captured_and_replayed():
    """Forward and backward in one graph, replayed on new inputs, while eager
    calls run between the replays."""
    x, dy, w, b = inputs(300, 1536, BF, 12)
    ws = torch.empty(m.lib().mxfp4_layernorm_backward_workspace(300, 1536), dtype=torch.uint8,
                     device="cuda")
    step = lambda: m.layernorm_backward(dy, x, *m.layernorm(x, w, b, want_stats=True)[1:], w,
                                        workspace=ws)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (13, 14):
        x2, dy2, _, _ = inputs(300, 1536, BF, seed)
        x.copy_(x2), dy.copy_(dy2)
        graph.replay()
        eager = m.layernorm_backward(dy2, x2, *m.layernorm(x2, w, b, want_stats=True)[1:], w)
        for a, c in zip(out, eager):
            assert torch.equal(a, c)


def test_two_streams_at_once():
    x, dy, w, b = inputs(2000, 1024, BF, 15)
    want = m.layernorm_backward(dy, x, *m.layernorm(x, w, b, want_stats=True)[1:], w)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        _, mean, rstd = m.layernorm(x, w, b, want_stats=True, stream=s)
        s.synchronize()
        with torch.cuda.stream(s):
            got.append(m.layernorm_backward(dy, x, mean, rstd, w))
    torch.cuda.synchronize()
    for g in got:
        for a, c in zip(g, want):
            assert torch.equal(a, c)


# more rows than a round of the persistent grid, at the widths where a thread
# holds most: one warp a row, several, a whole CTA, a cluster of two
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("shape", [(2500, 1024), (2500, 1023), (1500, 2563), (700, 4096),
                                   (701, 8192), (611, 8195), (611, 14336), (597, 14337),
                                   (350, 16384), (333, 24576), (310, 24577)])
def test_many_wide_rows(shape, dt):
    x, dy, w, b = inputs(*shape, dt, 12)
    x[-1] = 2.0
    x[3, -1] = float("inf")
    y, mean, rstd = m.layernorm(x, w, b, want_stats=True)
    assert torch.isnan(y[3]).all()
    keep = [i for i in range(shape[0]) if i != 3]
    check_forward(x[keep], w, b, 1e-5, y[keep], mean[keep], rstd[keep])
    if shape[1] % 32 == 0:
        codes, scales = m.layernorm_quantize(x, w, b)
        want = m.quantize(y)
        assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    x[3, -1] = 0.0
    y, mean, rstd = m.layernorm(x, w, b, want_stats=True)
    check_backward(dy, x, mean, rstd, w, *m.layernorm_backward(dy, x, mean, rstd, w))


# rows off the 16-byte boundary share a grid of whole groups of 8 (4) blocks;
# few rows leave some of them without any: one warp a row, several, a cluster,
# and more columns than a cluster holds
@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("rows", [1, 3, 5, 9, 33, 100, 197, 301, 595])
@pytest.mark.parametrize("cols", [5, 63, 1111, 4099, 9001, 16383, 70001])
def test_backward_stays_inside_its_workspace(rows, cols, dt):
    """A workspace of exactly the stated size: the bytes on both sides stay as
    they were, and what it held before does not matter."""
    if rows * cols > 6_000_000:
        rows = max(1, 6_000_000 // cols) | 1
    x, dy, w, b = inputs(rows, cols, dt, 16)
    _, mean, rstd = m.layernorm(x, w, b, want_stats=True)
    need = m.lib().mxfp4_layernorm_backward_workspace(rows, cols)
    pad = 16 * 8 * cols + 4096           # more than 8 partial rows [2][cols]
    buf = torch.full((256 + need + pad,), 0xFF, dtype=torch.uint8, device="cuda")
    out = m.layernorm_backward(dy, x, mean, rstd, w, workspace=buf[256:256 + need])
    torch.cuda.synchronize()
    assert (buf[:256] == 0xFF).all() and (buf[256 + need:] == 0xFF).all()
    check_backward(dy, x, mean, rstd, w, *out)


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("rows", [1, 6, 21])
def test_backward_of_shifted_tensors_stays_inside_its_workspace(rows, dt):
    """Whole vectors a row, but every tensor starts one element late."""
    cols = 256
    x, dy, w, b = inputs(rows, cols, dt, 17)
    late = [torch.zeros(rows * cols + 1, dtype=dt, device="cuda")[1:].view(rows, cols)
            for _ in range(3)]
    late[0].copy_(x), late[1].copy_(dy)
    _, mean, rstd = m.layernorm(x, w, b, want_stats=True)
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    need = m.lib().mxfp4_layernorm_backward_workspace(rows, cols)
    buf = torch.full((256 + need + 40 * cols * 8,), 0xFF, dtype=torch.uint8, device="cuda")
    m.layernorm_backward(late[1], late[0], mean, rstd, w, out=(late[2], dw, db),
                         workspace=buf[256:256 + need])
    torch.cuda.synchronize()
    assert (buf[:256] == 0xFF).all() and (buf[256 + need:] == 0xFF).all()
    check_backward(dy, x, mean, rstd, w, late[2], dw, db)


@pytest.mark.parametrize("dt,cols", [(F, 24576), (BF, 24576), (F, 14336), (BF, 14336)])
def test_clusters_that_start_apart(dt, cols):
    """Rows over two CTAs while products on another stream hold most of the
    SMs, which come free one after another: a row of each cluster is its
    first, and the same bits come out as on an idle GPU."""
    x, dy, w, b = inputs(200, cols, dt, 18)

    def work():
        y, mean, rstd = m.layernorm(x, w, b, want_stats=True)
        return (y, mean, rstd, *m.layernorm_backward(dy, x, mean, rstd, w))
    want = work()
    check_forward(x, w, b, 1e-5, *want[:3])
    check_backward(dy, x, want[1], want[2], w, *want[3:])
    side = torch.cuda.Stream()
    a = torch.randn(2048, 2048, device="cuda", dtype=BF)
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(side):
            for _ in range(6):
                a @ a
        got = work()
        for p, q in zip(got, want):
            assert torch.equal(p, q)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dt,wide,narrow", [(BF, 4096, 2048), (F, 2048, 1024), (F, 8192, 4112)])
def test_threads_take_turns_at_one_kernel(dt, wide, narrow):
    """One kernel asks for shared memory by the width of its rows. A second
    thread that comes to it with narrower rows takes nothing from the first."""
    import threading
    make = lambda cols: inputs(700, cols, dt, 19)
    (x, dy, w, b), (x2, dy2, w2, b2) = make(wide), make(narrow)

    def work(x, dy, w, b):
        y, mean, rstd = m.layernorm(x, w, b, want_stats=True)
        return (y, *m.layernorm_backward(dy, x, mean, rstd, w))
    want, want2 = work(x, dy, w, b), work(x2, dy2, w2, b2)
    want = work(x, dy, w, b)                 # this thread's last width: the wide one
    failures = []

    def other():
        try:
            for p, q in zip(work(x2, dy2, w2, b2), want2):
                assert torch.equal(p, q)
        except BaseException as e:           # noqa: B902 (reported below)
            failures.append(e)
    for _ in range(3):
        t = threading.Thread(target=other)   # a thread that has called nothing yet
        t.start()
        t.join()
        assert not failures, failures
        for p, q in zip(work(x, dy, w, b), want):
            assert torch.equal(p, q)


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("cols", [96, 1024, 17024])
def test_quantize_of_strided_and_unaligned_rows(dt, cols):
    """Rows of a wider tensor, on and off 16-byte boundaries, and dense rows
    that start one element late: the codes are those of the y that the same
    call writes, which is layernorm's."""
    x, _, w, b = inputs(30, 2 * cols + 8, dt, 20)
    w, b = w[:cols].clone(), b[:cols].clone()
    late = torch.zeros(30 * cols + 1, dtype=dt, device="cuda")[1:].view(30, cols)
    late.copy_(x[:, :cols])
    for xv in (x[::3, 8:cols + 8], x[:, 1:cols + 1], late):
        y, mean, rstd = m.layernorm(xv, w, b, want_stats=True)
        check_forward(xv, w, b, 1e-5, y, mean, rstd)
        codes, scales = m.quantize(y)
        got = m.layernorm_quantize(xv, w, b, want_y=True, want_stats=True)
        for p, q in zip(got, (codes, scales, y, mean, rstd)):
            assert torch.equal(p, q)
        alone = m.layernorm_quantize(xv, w, b)
        assert torch.equal(alone[0], codes) and torch.equal(alone[1], scales)
    # x and y equally late: each call has its own order of sums, and the codes
    # follow the y beside them
    out = torch.zeros(30 * cols + 1, dtype=dt, device="cuda")[1:].view(30, cols)
    got = m.layernorm_quantize(late, w, b, want_y=True, want_stats=True, out=(
        torch.empty(30, cols // 2, dtype=torch.uint8, device="cuda"),
        torch.empty(30, cols // 32, dtype=torch.uint8, device="cuda"), out, mean, rstd))
    check_forward(late, w, b, 1e-5, out, mean, rstd)
    codes, scales = m.quantize(out.clone())
    assert torch.equal(got[0], codes) and torch.equal(got[1], scales)
