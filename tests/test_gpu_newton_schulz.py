"""Newton-Schulz orthogonalization (mxfp4_newton_schulz) against the same
iteration in 64 bits.

One step is held to an elementwise bound. With r = 2^-11 / 2 (half a step of
fp16, the operands' type) and u = 2^-24 (fp32 sums of k terms): the operand
X16 is off by r |X|; A = X16 X16^T by at most (2 r + k u) |X||X|^T and, stored,
by r |A| more; B = b A + c A A by |b| dA + |c| (|A| dA + dA |A| + s u |A||A|)
and r |B|; X' = a X + B X16 by dB |X| + r |B||X| + s u |B||X|, the fp32
arithmetic of the epilogue and the output's own half step.

Several steps are held to the norm-wise form of that with each step's
amplification, the largest |f'| of f(s) = a s + b s^3 + c s^5 over the
singular values (that is the Lipschitz constant of the step in the Frobenius
norm). It is a loose bound (errors do not line up); what the steps do to each
singular value is checked on matrices whose arithmetic can be followed."""
import ctypes

import numpy as np
import pytest
import torch

import mxfp4_block_quantization_quantizer_b200 as m
from mxfp4_block_quantization_quantizer_b200 import build as B

pytestmark = pytest.mark.gpu

R, U = 2.0 ** -12, 2.0 ** -24
BF, F = torch.bfloat16, torch.float32
MUON = (3.4445, -4.7750, 2.0315)


def matrix(rows, cols, dt, seed, kind="normal"):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    if kind == "lowrank":
        r = max(1, min(rows, cols) // 16)
        x = 0.05 * x + torch.randn(rows, r, generator=g, device="cuda") @ torch.randn(
            r, cols, generator=g, device="cuda") / r ** 0.5
    return (0.01 * x).to(dt)


def start64(g, eps):
    x = g.double()
    return x / (x.square().sum().sqrt() + eps)


def step64(x, c):
    p = x @ x.T
    return c[0] * x + (c[1] * p + c[2] * (p @ p)) @ x


# tiles of 64 and 128 columns and of CTA pairs, single and ragged tiles, several
# tiles a CTA, wide and tall
SHAPES = [(1, 1), (1, 7), (9, 1), (64, 64), (128, 256), (130, 70), (33, 1000), (1000, 33),
          (257, 259), (300, 2049), (2050, 300), (512, 512), (1537, 1001), (1001, 1537),
          (1900, 4099), (4099, 1900), (2944, 2944), (520, 9000), (2304, 13000)]


@pytest.mark.parametrize("coeffs", [(0.0, 1.0, 0.0), (1.0, 0.0, 1.0), MUON])
@pytest.mark.parametrize("shape", SHAPES)
def test_one_step(shape, coeffs):
    g = matrix(*shape, F, 1)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = m.newton_schulz(g, 1, coeffs, out_dtype=F, status=st).double()
    assert int(st.item()) == 0
    x = start64(g, 1e-7)
    if shape[0] > shape[1]:
        x, got = x.T, got.T
    a, b, c = (abs(v) for v in coeffs)
    s, k = x.shape
    ax = x.abs()
    A = x @ x.T
    pa = ax @ ax.T
    dA = (2 * R + k * U + R) * pa * (1 + 4 * R)
    Bm = coeffs[1] * A + coeffs[2] * (A @ A)
    aA = A.abs()
    dB = b * dA + c * (aA @ dA + dA @ aA + dA @ dA + (s + 2) * U * aA @ aA)
    dB = dB + (R + 4 * U) * (Bm.abs() + dB)
    tol = dB @ ax + (R + (s + 2) * U) * (Bm.abs() + dB) @ ax + 8 * U * a * ax + 1e-9
    err = (got - step64(x, coeffs)).abs()
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("dt,out", [(BF, BF), (F, F), (F, BF), (BF, F)])
@pytest.mark.parametrize("shape,kind", [((256, 512), "normal"), ((200, 1000), "lowrank"),
                                        ((1000, 200), "lowrank"), ((513, 513), "normal")])
def test_several_steps(shape, kind, dt, out):
    g = matrix(*shape, dt, 2, kind)
    got = m.newton_schulz(g, 5, MUON, out_dtype=out)
    assert got.dtype == out
    a, b, c = MUON
    x = start64(g, 1e-7)
    if shape[0] > shape[1]:
        x, got = x.T, got.T
    err, s = 2.0 ** -21, x.shape[0]
    for _ in range(5):
        sv = torch.linalg.svdvals(x)
        top = torch.linspace(0, float(sv.max()), 4096, dtype=torch.float64)
        lip = float((a + 3 * b * top ** 2 + 5 * c * top ** 4).abs().max())
        x2, xf = float(sv.max()), float(sv.square().sum().sqrt())
        af = float((sv ** 4).sum().sqrt())
        bs = (b * sv ** 2 + c * sv ** 4).abs()
        dA = 2 * R * x2 * xf + R * af + x.shape[1] * U * xf * xf
        inj = R * float(bs.max()) * xf + R * float(bs.square().sum().sqrt()) * x2 \
            + (abs(b) + 2 * abs(c) * x2 ** 2) * dA * x2 + 8 * s * U * xf
        err = 1.05 * lip * err + inj
        x = step64(x, MUON)
    off = float((got.double() - x).norm())
    assert off <= err + 0.5 * torch.finfo(out).eps * float(x.norm())
    # what the iteration is for: singular values around 1
    sv = torch.linalg.svdvals(got.double())
    ref = torch.linalg.svdvals(x)
    assert (sv - ref).abs().max() <= err


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("shape", [(64, 64), (256, 640), (640, 256), (384, 300)])
def test_signed_permutations_follow_the_scalar_iteration(shape, dt):
    """G = a signed permutation of 64 entries, the rest zero: every product
    has one term, so each entry follows the scalar iteration with the same
    roundings (fp16 operands, two-half carry), bit for bit in fp32."""
    rows, cols = shape
    g = torch.zeros(rows, cols)
    rng = np.random.Generator(np.random.PCG64(3))
    ri, ci = rng.permutation(rows)[:64], rng.permutation(cols)[:64]
    sign = rng.choice([-1.0, 1.0], 64)
    g[ri, ci] = torch.tensor(sign, dtype=torch.float32)
    a, b, c = (np.float32(v) for v in (1.5, -0.75, 0.25))
    f, h = np.float32, np.float16
    x = f(4096.0 / 8)                       # times 2^12; |G|_F = 8, eps = 0
    for _ in range(6):
        hi = h(x)
        lo = h(f(x) - f(hi))
        A = h(f(hi) * f(hi) * f(2.0 ** -12))
        alpha = f(c * f(2.0 ** -12))
        Bv = h(f(np.float64(b) * float(f(A)) + float(f(alpha * f(f(A) * f(A))))))
        acc = f(f(Bv) * f(hi))
        x = f(np.float64(a) * float(f(hi) + f(lo)) + float(f(acc * f(2.0 ** -12))))
    want = torch.zeros(rows, cols)
    want[ri, ci] = torch.tensor(sign * float(f(x * f(2.0 ** -12))), dtype=torch.float32)
    got = m.newton_schulz(g.to(dt).cuda(), 6, (1.5, -0.75, 0.25), eps=0.0, out_dtype=F).cpu()
    assert torch.equal(got, want)


def test_scale_zero_and_special_inputs():
    g = matrix(100, 300, F, 4)
    base = m.newton_schulz(g, out_dtype=F)
    assert torch.equal(m.newton_schulz(g, scale=-0.5), -0.5 * base)
    z = m.newton_schulz(torch.zeros(100, 300, device="cuda"))
    assert (z == 0).all()
    # the norm is taken out: any power of two in G leaves the result alone
    # (eps = 0), far outside the range of fp32 squares
    one = m.newton_schulz(g, eps=0.0)
    for p in (2.0 ** 100, 2.0 ** -90):
        assert torch.equal(m.newton_schulz(g * p, eps=0.0), one)
    for bad in (float("nan"), float("inf")):
        h = g.clone()
        h[3, 5] = bad
        assert torch.isnan(m.newton_schulz(h)).all()


def test_in_place_and_output_bounds():
    for rows, cols, dt in ((65, 77, F), (300, 513, BF), (513, 300, BF)):
        g = matrix(rows, cols, dt, 5)
        want = m.newton_schulz(g)
        buf = torch.full((64 + rows * cols + 64,), 7.0, dtype=dt, device="cuda")
        m.newton_schulz(g, out=buf[64:-64].view(rows, cols))
        torch.cuda.synchronize()
        assert (buf[:64] == 7).all() and (buf[-64:] == 7).all()
        assert torch.equal(buf[64:-64].view(rows, cols), want)
        need = m.lib().mxfp4_newton_schulz_workspace(rows, cols)
        ws = torch.full((need + 512,), 0x7E, dtype=torch.uint8, device="cuda")  # fp16 NaN bytes
        out = m.newton_schulz(g, out=g, workspace=ws[:need])
        torch.cuda.synchronize()
        assert out is g and torch.equal(g, want) and (ws[need:] == 0x7E).all()


def test_captured_and_replayed():
    g = matrix(200, 500, BF, 6)
    ws = torch.empty(m.lib().mxfp4_newton_schulz_workspace(200, 500), dtype=torch.uint8,
                     device="cuda")
    m.newton_schulz(g, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.newton_schulz(g, workspace=ws)
    for seed in (7, 8):
        g.copy_(matrix(200, 500, BF, seed))
        want = m.newton_schulz(g.clone())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_two_streams_at_once():
    gs = [matrix(700, 900, F, s) for s in (9, 10)]
    want = [m.newton_schulz(g) for g in gs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in gs], []
    for s, g in zip(streams, gs):
        with torch.cuda.stream(s):
            got.append(m.newton_schulz(g))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_timeout_sets_status_and_poisons(tmp_path):
    """A build whose accumulator waits give up at once: NaN, the status bit,
    and an intact context."""
    path = str(tmp_path / "libmxfp4_shortwait.so")
    B.build_variant(path, ["MXFP4_ACC_WAIT_POLLS=0"])
    L = ctypes.CDLL(path)
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    L.mxfp4_newton_schulz.argtypes = [vp, i32, i64, i64, i32, f32, f32, f32, f32, f32, vp, i32,
                                      vp, i64, vp, vp]
    g = matrix(300, 400, F, 11)
    out = torch.zeros(300, 400, device="cuda")
    need = m.lib().mxfp4_newton_schulz_workspace(300, 400)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert L.mxfp4_newton_schulz(g.data_ptr(), m.F32, 300, 400, 2, *MUON, 1e-7, 1.0,
                                 out.data_ptr(), m.F32, ws.data_ptr(), need, st.data_ptr(),
                                 torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert int(st.item()) == m.STATUS_WAIT_TIMEOUT and torch.isnan(out).all()
    assert torch.isfinite(m.newton_schulz(g)).all()


def test_timeout_of_pairs_and_of_several_tiles(tmp_path):
    """The build whose accumulator waits give up at once, on matrices whose
    products run as CTA pairs (the last one of 2944 x 2944, all of 4096 x
    4096) and as several tiles of 128 x 128 a CTA (the first two of 2944): the
    warps that load operands stop wherever they are, and every load still
    lands before its CTA ends, in no more than a moment."""
    path = str(tmp_path / "libmxfp4_shortwait.so")
    B.build_variant(path, ["MXFP4_ACC_WAIT_POLLS=0"])
    L = ctypes.CDLL(path)
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    L.mxfp4_newton_schulz.argtypes = [vp, i32, i64, i64, i32, f32, f32, f32, f32, f32, vp, i32,
                                      vp, i64, vp, vp]
    for side in (2944, 4096):
        g = matrix(side, side, F, 12)
        want = m.newton_schulz(g, 1)
        out = torch.zeros_like(g)
        need = m.lib().mxfp4_newton_schulz_workspace(side, side)
        ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        for _ in range(5):
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            begin.record()
            assert L.mxfp4_newton_schulz(g.data_ptr(), m.F32, side, side, 1, *MUON, 1e-7, 1.0,
                                         out.data_ptr(), m.F32, ws.data_ptr(), need,
                                         st.data_ptr(),
                                         torch.cuda.current_stream().cuda_stream) == 0
            end.record()
            torch.cuda.synchronize()
            assert int(st.item()) == m.STATUS_WAIT_TIMEOUT and torch.isnan(out).all()
            # a wait for a load that never comes takes seconds
            assert begin.elapsed_time(end) < 500
            assert torch.equal(m.newton_schulz(g, 1), want)


def rounded64(x, c, steps):
    """The iteration in 64 bits with the operands' stated roundings: X carried
    as two fp16 values, A and B as one, all times 2^12."""
    h = lambda t: t.half().double()
    x = 4096 * x
    for _ in range(steps):
        hi = h(x)
        lo = h(x - hi)
        A = h(hi @ hi.T / 4096)
        Bm = h(c[1] * A + c[2] * (A @ A) / 4096)
        x = c[0] * (hi + lo) + Bm @ hi / 4096
    return x / 4096


@pytest.mark.parametrize("steps", [4, 5, 6])
@pytest.mark.parametrize("shape,kind", [
    (s, k) for s in [(64, 64), (64, 1000), (130, 70), (256, 512), (300, 2049), (1000, 200),
                     (513, 513), (1537, 1001), (96, 14336), (2944, 2944)]
    for k in ("normal", "lowrank")])
def test_error_is_that_of_the_stated_roundings(shape, kind, steps):
    """fp32 results against 64 bits, norm-wise: no further off than the header
    says (3e-3 for up to six steps, shorter side from 64 on), and no further
    than the roundings that it names take the same iteration. What the kernels
    add to those are fp32 sums, off by about sqrt(k) 2^-24, a thirtieth of an
    fp16 half step; but each such difference moves a later rounding by chance,
    so the two errors are of one size and not the same: half as much again
    bounds the difference of two norms of thousands of such roundings."""
    g = matrix(*shape, F, 13, kind)
    got = m.newton_schulz(g, steps, MUON, out_dtype=F).double()
    x = start64(g, 1e-7)
    if shape[0] > shape[1]:
        x, got = x.T, got.T
    near = rounded64(x, MUON, steps)
    for _ in range(steps):
        x = step64(x, MUON)
    norm = float(x.norm())
    off, model = float((got - x).norm()) / norm, float((near - x).norm()) / norm
    assert off <= 3e-3 and off <= 1.5 * model + 2.0 ** -20, (off, model)


@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (9, 1), (3, 5), (16, 16), (33, 1000),
                                   (1000, 33)])
def test_error_of_few_singular_values(shape):
    """A shorter side below 64: the header's 1e-2 for five steps. (A step moves
    a singular value by up to 1e-3 through the roundings of A and B, and the
    steps that follow, with |f'| up to 1.3 around 1, multiply that.)"""
    for seed in range(5):
        g = matrix(*shape, F, 14 + seed)
        got = m.newton_schulz(g, 5, MUON, out_dtype=F).double()
        x = start64(g, 1e-7)
        if shape[0] > shape[1]:
            x, got = x.T, got.T
        for _ in range(5):
            x = step64(x, MUON)
        assert float((got - x).norm()) <= 1e-2 * float(x.norm())
