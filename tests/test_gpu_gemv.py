"""Products of bf16 rows with an MXFP4 weight (mxfp4_gemv) against the same
sum in 64 bits.

Bound, with u = 2^-24: a bf16 x enters as eight E2M1 digits whose sum is off
by at most 2^-23 of the largest magnitude in its group of 32 (and exact where
|x| is at least 2^-16 of it). Every product of a code and a digit is exact.
The digits' magnitudes add up to at most |x| (1 + 1/4) (a digit leaves at most
half a step, below a fifth of itself), so the 8 k products, added in fp32 in
some order, are off by at most (k + 64) u of 1.25 sum |x| |w|: k - 1 additions
in each of the digits' columns, then the joining of columns and slabs. An
output is rounded once, by at most half a step of its type.
"""
import ctypes

import numpy as np
import pytest
import torch

import mxfp4_block_quantization_quantizer_b200 as m
from mxfp4_block_quantization_quantizer_b200 import build as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def weight(n, k, seed, lo=100, hi=140):
    """Every code, scale bytes in [lo, hi)."""
    g = gen(seed)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(lo, hi, (n, k // 32), generator=g, device="cuda", dtype=torch.uint8)
    return codes, scales


def values(codes, scales, n, k):
    return m.dequantize(codes, scales, n, k, m.ROWS, F).double()


def check(y, x, codes, scales):
    rows, k = x.shape
    n = codes.shape[0]
    w = values(codes, scales, n, k)
    xd = x.double()
    gmax = xd.abs().reshape(rows, k // 32, 32).amax(-1).repeat_interleave(32, 1)
    want = xd @ w.T
    # (scale bytes end at 2^-127: groups below 2^-104 keep multiples of 2^-128)
    off = torch.where(gmax < 2.0 ** -104, torch.full_like(gmax, 2.0 ** -128), 2.0 ** -23 * gmax)
    tol = (k + 64) * U * 1.25 * (xd.abs() @ w.abs().T) + off @ w.abs().T
    tol = tol + 0.5 * torch.finfo(y.dtype).eps * (want.abs() + tol) + 1e-37
    err = (y.double() - want).abs()
    assert torch.isfinite(y).all()
    assert (err <= tol).all(), (err / tol).max()


# 1 to 8 slabs of k; tiles of 2, 8, 16 and 32 tokens; ragged n; k that ends
# inside a stage (256), a scale tile (128) and an MMA (64)
SHAPES = [(1, 128, 128), (1, 1, 128), (2, 130, 256), (1, 4096, 4096), (3, 1000, 512),
          (8, 384, 1536), (9, 257, 640), (16, 4096, 1024), (17, 100, 2048), (32, 640, 896),
          (33, 129, 1280), (64, 512, 768), (65, 200, 384), (150, 260, 512), (5, 20000, 256),
          (1, 40000, 128), (4, 128, 28672),
          (1, 77, 32), (1, 300, 96), (7, 65, 160), (8, 128, 4128), (37, 1537, 1440), (20, 9, 64)]


@pytest.mark.parametrize("out", [BF, F])
@pytest.mark.parametrize("shape", SHAPES)
def test_products(shape, out):
    rows, n, k = shape
    codes, scales = weight(n, k, 1)
    x = torch.randn(rows, k, generator=gen(2), device="cuda").to(BF)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    blocked = m.scales_to_blocked(scales)
    y = m.gemv(x, codes, blocked, out_dtype=out, status=st)
    assert int(st.item()) == 0 and y.dtype == out and y.shape == (rows, n)
    check(y, x, codes, scales)
    assert torch.equal(y, m.gemv(x, codes, blocked, out_dtype=out))   # the same bits again


@pytest.mark.parametrize("rows,k", [(1, 1024), (16, 1024), (40, 512), (3, 96)])
def test_whole_numbers_are_exact(rows, k):
    """x whole below 2^8 (exact digits), scales 1: every partial sum of a
    digit's column is a multiple of 2^-16 of less than 24 bits or cancels
    exactly, so no addition rounds."""
    codes, _ = weight(192, k, 3)
    scales = torch.full((192, k // 32), 127, dtype=torch.uint8, device="cuda")
    x = torch.randint(-255, 256, (rows, k), generator=gen(4), device="cuda").to(BF)
    y = m.gemv(x, codes, m.scales_to_blocked(scales), out_dtype=F)
    assert torch.equal(y.double(), x.double() @ values(codes, scales, 192, k).T)


@pytest.mark.parametrize("k", [512, 160])
def test_one_token_moves_one_row(k):
    """A single non-zero x picks one column of the weight, exactly, at every
    position of a k block and for tokens in both halves of a tile."""
    codes, scales = weight(130, k, 5, 120, 131)
    w = values(codes, scales, 130, k)
    blocked = m.scales_to_blocked(scales)
    x = torch.zeros(24, k, dtype=BF, device="cuda")
    at = [(7 * t + 33 * (t % 5) + t * t) % k for t in range(24)]
    for t, c in enumerate(at):
        x[t, c] = 1.0 + t / 32        # up to 6 significant bits
    y = m.gemv(x, codes, blocked, out_dtype=F).double()
    assert torch.equal(y, torch.stack([w[:, c] * (1 + t / 32) for t, c in enumerate(at)]))


@pytest.mark.parametrize("spread", [6, 13, 30])
def test_wide_ranges_inside_a_group(spread):
    """Magnitudes of one group 2^spread apart, and outliers of 2^10."""
    codes, scales = weight(256, 1024, 6)
    g = gen(7)
    x = torch.randn(10, 1024, generator=g, device="cuda")
    x = x * torch.exp2(-spread * torch.rand(10, 1024, generator=g, device="cuda"))
    x[:, ::97] *= 1024
    x = x.to(BF)
    check(m.gemv(x, codes, m.scales_to_blocked(scales), out_dtype=F), x, codes, scales)


def test_small_x_beside_a_large_one_with_zero_weight():
    """Where |x| is at least 2^-16 of its group's maximum its digits are exact:
    an outlier that meets zero codes costs its neighbours nothing."""
    codes = torch.full((128, 128), 0x22, dtype=torch.uint8, device="cuda")   # all 1.0
    codes[:, 0] = 0x20                                                       # k = 0: code 0
    scales = torch.full((128, 8), 127, dtype=torch.uint8, device="cuda")
    x = torch.zeros(1, 256, dtype=BF, device="cuda")
    x[0, 0] = 2.0 ** 12
    x[0, 1:32] = 0.50390625 + torch.arange(31, device="cuda") / 256    # 8 significant bits
    x = x.to(BF)
    y = m.gemv(x, codes, m.scales_to_blocked(scales), out_dtype=F)
    assert (y.double() == x[0, 1:].double().sum()).all()


@pytest.mark.parametrize("byte_x,byte_w", [(2.0 ** 60, 60), (2.0 ** -60, 190), (2.0 ** -126, 200),
                                           (2.0 ** -130, 245), (2.0 ** 100, 20)])
def test_far_scales(byte_x, byte_w):
    codes, scales = weight(140, 256, 8, byte_w, byte_w + 3)
    x = (torch.randn(4, 256, generator=gen(9), device="cuda").double() * byte_x).to(BF)
    check(m.gemv(x, codes, m.scales_to_blocked(scales), out_dtype=F), x, codes, scales)


@pytest.mark.parametrize("k", [512, 544])
def test_nonfinite_groups(k):
    codes, scales = weight(140, k, 10)
    x = torch.randn(12, k, generator=gen(11), device="cuda").to(BF)
    clean = m.gemv(x, codes, m.scales_to_blocked(scales))
    x[3, 40], x[10, 1] = float("nan"), float("nan")
    scales[77, 2] = 0xFF
    y = m.gemv(x, codes, m.scales_to_blocked(scales))
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[3], bad[10] = True, True
    bad[:, 77] = True
    assert torch.equal(torch.isnan(y), bad)
    assert torch.equal(y[~bad], clean[~bad])
    x[3, 40] = float("inf")
    y = m.gemv(x, codes, m.scales_to_blocked(scales))
    assert not torch.isfinite(y[3]).any() and torch.equal(y[~bad], clean[~bad])


def test_strided_rows_and_unaligned_codes():
    codes, scales = weight(200, 512, 12)
    blocked = m.scales_to_blocked(scales)
    wide = torch.randn(30, 1536, generator=gen(13), device="cuda").to(BF)
    x = wide[::3, 512:1024]
    want = m.gemv(x.contiguous(), codes, blocked)
    assert torch.equal(m.gemv(x, codes, blocked), want)
    # codes off a 32-byte boundary
    raw = torch.zeros(codes.numel() + 64, dtype=torch.uint8, device="cuda")
    off = raw[16:16 + codes.numel()].view(200, 256)
    off.copy_(codes)
    y = m.gemv(x, off, blocked, out_dtype=F)
    check(y, x, codes, scales)


def test_quantizer_outputs_and_row_slices():
    """A weight straight from the quantizer, and 128 rows of it."""
    w = 0.02 * torch.randn(512, 1024, generator=gen(14), device="cuda")
    codes, scales = m.quantize(w)
    x = torch.randn(2, 1024, generator=gen(15), device="cuda").to(BF)
    y = m.gemv(x, codes, m.scales_to_blocked(scales), out_dtype=F)
    check(y, x, codes, scales)
    part = m.gemv(x, codes[128:256], m.scales_to_blocked(scales[128:256]), out_dtype=F)
    check(part, x, codes[128:256], scales[128:256])


@pytest.mark.parametrize("rows,n,k", [(3, 130, 512), (70, 257, 256), (5, 77, 96)])
def test_output_ends_where_it_should(rows, n, k):
    codes, scales = weight(n, k, 16)
    x = torch.randn(rows, k, generator=gen(17), device="cuda").to(BF)
    for dt in (BF, F):
        buf = torch.full((64 + rows * n + 64,), 7.0, dtype=dt, device="cuda")
        m.gemv(x, codes, m.scales_to_blocked(scales), out=buf[64:-64].view(rows, n))
        torch.cuda.synchronize()
        assert (buf[:64] == 7).all() and (buf[-64:] == 7).all()


def test_captured_and_replayed_on_another_stream():
    codes, scales = weight(1024, 2048, 18)
    blocked = m.scales_to_blocked(scales)
    x = torch.randn(4, 2048, generator=gen(19), device="cuda").to(BF)
    m.gemv(x, codes, blocked)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y = m.gemv(x, codes, blocked)
    for seed in (20, 21):
        x.copy_(torch.randn(4, 2048, generator=gen(seed), device="cuda"))
        want = m.gemv(x.clone(), codes, blocked)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_timeout_sets_status_and_poisons(tmp_path):
    """A build whose accumulator waits give up at once: NaN outputs, the
    status bit, and an intact context."""
    path = str(tmp_path / "libmxfp4_shortwait.so")
    B.build_variant(path, ["MXFP4_ACC_WAIT_POLLS=0"])
    L = ctypes.CDLL(path)
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    L.mxfp4_gemv.argtypes = [vp, i64, i64, i64, i64, vp, vp, vp, ctypes.c_int, vp, i64, vp, vp]
    for rows, n, k in ((2, 256, 1024), (9, 20000, 128)):
        codes, scales = weight(n, k, 22)
        blocked = m.scales_to_blocked(scales)
        x = torch.randn(rows, k, generator=gen(23), device="cuda").to(BF)
        y = torch.zeros(rows, n, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        need = m.lib().mxfp4_gemv_workspace(rows, n, k)
        ws = torch.zeros(need + 16, dtype=torch.uint8, device="cuda")
        assert L.mxfp4_gemv(x.data_ptr(), rows, n, k, k, codes.data_ptr(), blocked.data_ptr(),
                            y.data_ptr(), m.F32, ws.data_ptr(), need, st.data_ptr(),
                            torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert int(st.item()) == m.STATUS_WAIT_TIMEOUT and torch.isnan(y).all()
        check(m.gemv(x, codes, blocked, out_dtype=F), x, codes, scales)
