"""Refusals of the weight product, the layer norm and the Newton-Schulz update:
the C ABI rejects bad arguments with the documented status before any launch,
and the binding rejects bad tensors before any library call. CPU only."""
import ctypes

import pytest
import torch

import mxfp4_block_quantization_quantizer_b200 as m
from mxfp4_block_quantization_quantizer_b200 import _binding as B

OK, NULL, SHAPE, ALIGN, ENUM, CUDA, VALUE, WORKSPACE = range(8)
P = ctypes.c_void_p(4096)
P2 = ctypes.c_void_p(4096 + 2)
P8 = ctypes.c_void_p(4096 + 8)
P16 = ctypes.c_void_p(4096 + 16)
NUL = ctypes.c_void_p(0)
BIG = 1 << 60


def test_status_strings():
    texts = [m.status_string(s) for s in range(8)]
    assert len(set(texts)) == 8 and "unknown status" not in texts


@pytest.mark.parametrize("args,want", [
    ((NUL, 1, 256, 512, 512, P, P, P, 1, P, BIG, NUL), NULL),
    ((P, 1, 256, 512, 512, NUL, P, P, 1, P, BIG, NUL), NULL),
    ((P, 1, 256, 512, 512, P, NUL, P, 1, P, BIG, NUL), NULL),
    ((P, 1, 256, 512, 512, P, P, NUL, 1, P, BIG, NUL), NULL),
    ((P, 3, 256, 512, 512, P, P, P, 1, NUL, BIG, NUL), NULL),   # needs a workspace
    ((P, 1, 256, 512, 512, P, P, P, 2, P, BIG, NUL), ENUM),
    ((P, 0, 256, 512, 512, P, P, P, 1, P, BIG, NUL), SHAPE),
    ((P, 1, 0, 512, 512, P, P, P, 1, P, BIG, NUL), SHAPE),
    ((P, 1, 256, 0, 0, P, P, P, 1, P, BIG, NUL), SHAPE),
    ((P, 1, 256, 48, 48, P, P, P, 1, P, BIG, NUL), SHAPE),      # k % 32
    ((P, 2, 256, 512, 504, P, P, P, 1, P, BIG, NUL), SHAPE),    # rows overlap
    ((P, 2, 256, 512, 516, P, P, P, 1, P, BIG, NUL), SHAPE),    # stride % 8
    ((P, (1 << 19) + 1, 256, 512, 512, P, P, P, 1, P, BIG, NUL), SHAPE),
    ((P, 1, 32, 1 << 31, 1 << 31, P, P, P, 1, P, BIG, NUL), SHAPE),
    ((P8, 1, 256, 512, 512, P, P, P, 1, P, BIG, NUL), ALIGN),
    ((P, 1, 256, 512, 512, P8, P, P, 1, P, BIG, NUL), ALIGN),
    ((P, 1, 256, 512, 512, P, P8, P, 1, P, BIG, NUL), ALIGN),
    ((P, 1, 256, 512, 512, P, P, P8, 1, P, BIG, NUL), ALIGN),
    ((P, 3, 256, 512, 512, P, P, P, 1, P8, BIG, NUL), ALIGN),
    ((P, 1, 256, 512, 512, P, P, P, 1, P, BIG, P2), ALIGN),
    ((P, 3, 256, 512, 512, P, P, P, 1, P, 100, NUL), WORKSPACE),
])
def test_gemv_rejects_bad_arguments(args, want):
    assert m.lib().mxfp4_gemv(*args, NUL) == want


def test_workspace_sizes():
    L = m.lib()
    assert L.mxfp4_gemv_workspace(1, 4096, 4096) == 0
    assert L.mxfp4_gemv_workspace(2, 4096, 4096) == 0
    # eight digits of half a byte per x and their scales, rows padded to 8
    assert L.mxfp4_gemv_workspace(3, 1, 256) == 8 * (8 * 128) + 1024
    assert L.mxfp4_gemv_workspace(1, 4096, 48) == -1
    assert L.mxfp4_gemv_workspace(0, 4096, 64) == -1
    assert L.mxfp4_layernorm_backward_workspace(3, 10) == 3 * 2 * 10 * 4
    assert L.mxfp4_layernorm_backward_workspace(1 << 20, 10) == 592 * 2 * 10 * 4
    assert L.mxfp4_layernorm_backward_workspace(0, 10) == -1
    assert L.mxfp4_newton_schulz_workspace(100, 300) == L.mxfp4_newton_schulz_workspace(100, 300)
    assert L.mxfp4_newton_schulz_workspace(100, 300) >= 6 * 100 * 300 + 4 * 100 * 100
    assert L.mxfp4_newton_schulz_workspace(0, 300) == -1
    assert L.mxfp4_newton_schulz_workspace((1 << 20) + 1, 300) == -1


@pytest.mark.parametrize("args,want", [
    ((NUL, 1, 4, 64, 64, P, P, 1e-5, P, P, P), NULL),
    ((P, 1, 4, 64, 64, P, P, 1e-5, NUL, P, P), NULL),
    ((P, 2, 4, 64, 64, P, P, 1e-5, P, P, P), ENUM),
    ((P, 1, 0, 64, 64, P, P, 1e-5, P, P, P), SHAPE),
    ((P, 1, 4, 0, 64, P, P, 1e-5, P, P, P), SHAPE),
    ((P, 1, 4, 64, 63, P, P, 1e-5, P, P, P), SHAPE),
    ((P, 1, 1 << 32, 64, 64, P, P, 1e-5, P, P, P), SHAPE),
    ((P, 1, 1 << 20, 64, 1 << 40, P, P, 1e-5, P, P, P), SHAPE),
    ((P, 1, 4, 64, 64, P, P, -1.0, P, P, P), VALUE),
    ((P, 1, 4, 64, 64, P, P, float("nan"), P, P, P), VALUE),
    ((P, 1, 4, 64, 64, P, P, float("inf"), P, P, P), VALUE),
    ((P2, 0, 4, 64, 64, P, P, 1e-5, P, P, P), ALIGN),           # fp32 needs 4 bytes
    ((P, 1, 4, 64, 64, P2, P, 1e-5, P, P, P), ALIGN),
    ((P, 1, 4, 64, 64, P, P, 1e-5, P, P2, P), ALIGN),
])
def test_layernorm_rejects_bad_arguments(args, want):
    assert m.lib().mxfp4_layernorm(*args, NUL) == want


def test_layernorm_quantize_and_backward_reject_bad_arguments():
    L = m.lib()
    q = L.mxfp4_layernorm_quantize
    assert q(P, 1, 4, 64, 64, P, P, 1e-5, NUL, NUL, NUL, NUL, P, NUL) == NULL
    assert q(P, 1, 4, 64, 64, P, P, 1e-5, NUL, NUL, NUL, P, NUL, NUL) == NULL
    assert q(P, 1, 4, 80, 80, P, P, 1e-5, NUL, NUL, NUL, P, P, NUL) == SHAPE   # cols % 32
    assert q(P, 1, 4, 64, 64, P, P, 1e-5, NUL, NUL, NUL, P8, P, NUL) == ALIGN
    b = L.mxfp4_layernorm_backward
    good = (P, P, 1, 4, 64, 64, 64, P, P, P, P, P, P, P, BIG, NUL)

    def but(**kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return b(*a)
    for i in (0, 1, 8, 9, 10):
        assert but(**{"_%d" % i: NUL}) == NULL
    assert but(_11=NUL) == NULL and but(_12=NUL) == NULL     # dw without db, db without dw
    assert but(_13=NUL) == NULL                              # dw and db without workspace
    assert but(_2=3) == ENUM
    assert but(_5=63) == SHAPE and but(_6=63) == SHAPE
    assert but(_13=P8) == ALIGN
    assert but(_14=4 * 2 * 64 * 4 - 1) == WORKSPACE


@pytest.mark.parametrize("kw,want", [
    (dict(g=NUL), NULL), (dict(out=NUL), NULL), (dict(ws=NUL), NULL),
    (dict(dt=2), ENUM), (dict(odt=-1), ENUM),
    (dict(rows=0), SHAPE), (dict(cols=(1 << 20) + 1), SHAPE),
    (dict(steps=0), VALUE), (dict(steps=1001), VALUE), (dict(eps=-1e-9), VALUE),
    (dict(a=float("nan")), VALUE), (dict(c=2e4), VALUE), (dict(scale=float("inf")), VALUE),
    (dict(g=P8), ALIGN), (dict(out=P8), ALIGN), (dict(ws=P16), ALIGN), (dict(status=P2), ALIGN),
    (dict(bytes=1000), WORKSPACE),
])
def test_newton_schulz_rejects_bad_arguments(kw, want):
    d = dict(g=P, dt=1, rows=64, cols=96, steps=5, a=3.4, b=-4.7, c=2.0, eps=1e-7, scale=1.0,
             out=P, odt=1, ws=P, bytes=BIG, status=NUL, stream=NUL)
    d.update(kw)
    assert m.lib().mxfp4_newton_schulz(*d.values()) == want


@pytest.fixture
def fake(monkeypatch):
    calls = []
    monkeypatch.setattr(B, "_on_device", lambda t, name, device=None: None)
    monkeypatch.setattr(B, "_call", lambda name, device, stream, *a: calls.append(name))
    return calls


BF, F, U8 = torch.bfloat16, torch.float32, torch.uint8


def test_host_tensors_are_refused():
    x = torch.zeros(2, 64, dtype=BF)
    for f in (lambda: m.layernorm(x), lambda: m.layernorm_quantize(x), lambda: m.newton_schulz(x),
              lambda: m.gemv(x, torch.zeros(4, 32, dtype=U8), torch.zeros(128, 4, dtype=U8)),
              lambda: m.layernorm_backward(x, x, torch.zeros(2), torch.ones(2))):
        with pytest.raises(TypeError):
            f()


def test_gemv_checks_its_tensors(fake):
    x, c, s = torch.zeros(3, 256, dtype=BF), torch.zeros(20, 128, dtype=U8), torch.zeros(
        128, 8, dtype=U8)
    assert m.gemv(x, c, s).shape == (3, 20) and m.gemv(x, c, s, out_dtype=F).dtype == F
    wide = torch.zeros(6, 512, dtype=BF)
    m.gemv(wide[::2, 256:], c, s)
    n = len(fake)
    bad = [lambda: m.gemv(x.float(), c, s), lambda: m.gemv(x[0], c, s),
           lambda: m.gemv(wide[:, ::2], c, s), lambda: m.gemv(x, c[:, :64], s),
           lambda: m.gemv(x, c, s[:64]), lambda: m.gemv(x, c.int(), s),
           lambda: m.gemv(x, c, s, out=torch.zeros(3, 19, dtype=BF)),
           lambda: m.gemv(x, c, s, out=torch.zeros(20, 3, dtype=F).T),
           lambda: m.gemv(x, c, s, out_dtype=torch.float16),
           lambda: m.gemv(x, c, s, workspace=torch.zeros(8, dtype=U8)),
           lambda: m.gemv(x, c, s, status=torch.zeros(2, dtype=torch.int32)),
           lambda: m.gemv(x[:1].expand(3, 256), c, s)]
    for f in bad:
        with pytest.raises((TypeError, ValueError)):
            f()
    buf = torch.zeros(4000, dtype=BF)   # an output inside the input
    with pytest.raises(ValueError):
        m.gemv(buf[:768].view(3, 256), c, s, out=buf[700:760].view(3, 20))
    assert len(fake) == n


def test_layernorm_checks_its_tensors(fake):
    x, w, st = torch.zeros(4, 96, dtype=BF), torch.ones(96), torch.zeros(4)
    assert m.layernorm(x).shape == (4, 96)
    y, mean, rstd = m.layernorm(x, w, w, want_stats=True)
    assert mean.shape == (4,) and mean.dtype == F
    assert len(m.layernorm_quantize(x, w, want_y=True, want_stats=True)) == 5
    dx, dw, db = m.layernorm_backward(x, x, st, st, w)
    assert dw.shape == (96,) and dw.dtype == F
    assert m.layernorm_backward(x, x, st, st, want_params=False).shape == (4, 96)
    n = len(fake)
    for f in (lambda: m.layernorm(x.half()), lambda: m.layernorm(x[0]),
              lambda: m.layernorm(x.T), lambda: m.layernorm(x, w[:95]),
              lambda: m.layernorm(x, w.to(BF)), lambda: m.layernorm(x, out=x),
              lambda: m.layernorm(x, out=torch.zeros(4, 96)),
              lambda: m.layernorm(x[:1].expand(4, 96)),
              lambda: m.layernorm(x, want_stats=True, out=(y, mean, rstd[:3])),
              lambda: m.layernorm_quantize(x, out=(torch.zeros(4, 47, dtype=U8),
                                                   torch.zeros(4, 3, dtype=U8))),
              lambda: m.layernorm_quantize(x, want_y=True,
                                           out=(torch.zeros(4, 48, dtype=U8),
                                                torch.zeros(4, 3, dtype=U8))),
              lambda: m.layernorm_backward(x.float(), x, st, st),
              lambda: m.layernorm_backward(x[:3], x, st, st),
              lambda: m.layernorm_backward(x, x, st[:3], st),
              lambda: m.layernorm_backward(x, x, st, st, out=(x, w, w)),
              lambda: m.layernorm_backward(x, x, st, st, workspace=torch.zeros(5, dtype=U8))):
        with pytest.raises((TypeError, ValueError)):
            f()
    assert len(fake) == n


def test_newton_schulz_checks_its_tensors(fake):
    g = torch.zeros(20, 30)
    assert m.newton_schulz(g).dtype == F and m.newton_schulz(g, out_dtype=BF).dtype == BF
    assert m.newton_schulz(g, out=g) is g
    n = len(fake)
    for f in (lambda: m.newton_schulz(g.half()), lambda: m.newton_schulz(g.T),
              lambda: m.newton_schulz(g[0]), lambda: m.newton_schulz(g, out=g[:, :29]),
              lambda: m.newton_schulz(g, out=g.view(BF)[:, :30]),
              lambda: m.newton_schulz(g, workspace=torch.zeros(100, dtype=U8)),
              lambda: m.newton_schulz(g, out_dtype=torch.float16)):
        with pytest.raises((TypeError, ValueError)):
            f()
    assert len(fake) == n


def carve(*sizes, gap=256):
    """Disjoint byte ranges of one buffer, and the whole buffer."""
    whole = torch.zeros(sum(-(-n // gap) * gap + gap for n in sizes), dtype=U8)
    parts, at = [], 0
    for n in sizes:
        parts.append(whole[at:at + n])
        at += -(-n // gap) * gap + gap
    return whole, parts


def test_written_memory_that_meets_another_argument_is_refused(fake):
    """Every pair of a written tensor and another one that would be read or
    written beside it: apart it is taken, sharing bytes it is refused."""
    L = m.lib()

    def each(call, args, written, allowed=()):
        """args: name -> (bytes, function from a byte slice to the argument)."""
        whole, parts = carve(*(n for n, _ in args.values()))
        good = {k: f(p) for (k, (n, f)), p in zip(args.items(), parts)}
        call(**good)
        n = len(fake)
        place = dict(zip(args, parts))
        for a in written:
            for b in args:
                if a == b or (a, b) in allowed or (b, a) in allowed:
                    continue
                # a's bytes where b's last ones are, so that one byte meets
                size, f = args[a]
                end = place[b].data_ptr() - whole.data_ptr() + args[b][0]
                step = 4
                big = torch.zeros(end - step + size + 256, dtype=U8)
                big_b = args[b][1](big[end - args[b][0]:end])
                big_a = f(big[end - step:end - step + size])
                with pytest.raises(ValueError, match="overlaps"):
                    call(**{**good, b: big_b, a: big_a})
        assert len(fake) == n
    view = lambda t, *shape: (lambda s: s.view(t).view(*shape))
    R, C, K, N = 4, 96, 256, 20
    ln = dict(x=(R * C * 4, view(F, R, C)), weight=(C * 4, view(F, C)), bias=(C * 4, view(F, C)))
    stats = dict(mean=(R * 4, view(F, R)), rstd=(R * 4, view(F, R)))
    y = dict(y=(R * C * 4, view(F, R, C)))
    each(lambda x, weight, bias, y, mean, rstd: m.layernorm(x, weight, bias, want_stats=True,
                                                            out=(y, mean, rstd)),
         {**ln, **y, **stats}, ("y", "mean", "rstd"))
    q = dict(codes=(R * C // 2, view(U8, R, C // 2)), scales=(R * C // 32, view(U8, R, C // 32)))
    each(lambda x, weight, bias, codes, scales, y, mean, rstd:
         m.layernorm_quantize(x, weight, bias, want_y=True, want_stats=True,
                              out=(codes, scales, y, mean, rstd)),
         {**ln, **q, **y, **stats}, ("codes", "scales", "y", "mean", "rstd"))
    ws = L.mxfp4_layernorm_backward_workspace(R, C)
    back = dict(dy=ln["x"], x=ln["x"], weight=ln["weight"], **stats, dx=y["y"],
                dw=(C * 4, view(F, C)), db=(C * 4, view(F, C)), ws=(ws, view(U8, ws)))
    # dw and db are written when the inputs have been read
    late = [(a, b) for a in ("dw", "db") for b in ("dy", "x", "weight", "mean", "rstd")]
    each(lambda dy, x, weight, mean, rstd, dx, dw, db, ws:
         m.layernorm_backward(dy, x, mean, rstd, weight, out=(dx, dw, db), workspace=ws),
         back, ("dx", "dw", "db", "ws"), late)
    ws = L.mxfp4_gemv_workspace(3, N, K)
    each(lambda x, codes, blocked, out, ws, st: m.gemv(x, codes, blocked, out=out, workspace=ws,
                                                       status=st),
         dict(x=(3 * K * 2, view(BF, 3, K)), codes=(N * K // 2, view(U8, N, K // 2)),
              blocked=(128 * 8, view(U8, 128, 8)), out=(3 * N * 4, view(F, 3, N)),
              ws=(ws, view(U8, ws)), st=(4, view(torch.int32, 1))), ("out", "ws", "st"))
    ws = L.mxfp4_newton_schulz_workspace(R, C)
    each(lambda g, out, ws, st: m.newton_schulz(g, out=out, workspace=ws, status=st),
         dict(g=(R * C * 4, view(F, R, C)), out=(R * C * 4, view(F, R, C)), ws=(ws, view(U8, ws)),
              st=(4, view(torch.int32, 1))), ("out", "ws", "st"))


def test_what_lies_behind_a_workspace_of_more_than_enough_bytes_is_free(fake):
    """A workspace may be longer than a call needs, and tensors may lie in the
    rest of it."""
    L = m.lib()
    x, st = torch.zeros(4, 96), torch.zeros(4)
    need = L.mxfp4_layernorm_backward_workspace(4, 96)
    arena = torch.zeros(need + 4 * 96 * 4, dtype=U8)
    tail = arena[need:].view(F).view(4, 96)
    m.layernorm_backward(x, x, st, st, out=(tail, torch.zeros(96), torch.zeros(96)),
                         workspace=arena)
    need = L.mxfp4_newton_schulz_workspace(4, 96)
    arena = torch.zeros(need + 4 * 96 * 4, dtype=U8)
    m.newton_schulz(x, out=arena[need:].view(F).view(4, 96), workspace=arena)
    c, s = torch.zeros(20, 128, dtype=U8), torch.zeros(128, 8, dtype=U8)
    need = L.mxfp4_gemv_workspace(3, 20, 256)
    arena = torch.zeros(need + 3 * 20 * 4, dtype=U8)
    m.gemv(torch.zeros(3, 256, dtype=BF), c, s, out=arena[need:].view(F).view(3, 20),
           workspace=arena)
    assert len(fake) == 3
