"""The operators around a block-quantized linear layer, as measured cases.

- gemv: y = x W^T for a few bf16 activation rows x and an MXFP4 weight W
  (E2M1 codes with one power-of-two scale per 32 elements along k), the
  product a model answers single tokens with;
- ln_fwd, ln_bwd: the layer norm in front of a quantized linear layer, and
  its gradients (of the input, the gain and the offset);
- ns: a weight's update made nearly orthogonal by Newton-Schulz products,
  before the update reaches the master weight that the quantizer follows.

Each has a plain form in torch operations (run with own = False) and its call
of the package (own = True). The plain forms compute in 32 bits and round once
at the end; exact() computes the same definitions in 64 bits, written apart.
"""
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
NS_COEFFS = (3.4445, -4.7750, 2.0315)
NS_EPS = 1e-7
LN_EPS = 1e-6


def listed():
    return [
        # one token through a square projection: latency counts
        dict(name="gemv 1 4096x4096", op="gemv", m=1, n=4096, k=4096, out="bf16"),
        # one token through the largest weight
        dict(name="gemv 1 8192x28672", op="gemv", m=1, n=8192, k=28672, out="bf16"),
        # a batch of 16 tokens through an LLM weight, sums kept in 32 bits
        dict(name="gemv 16 4096x14336", op="gemv", m=16, n=4096, k=14336, out="f32"),
        # a ragged batch and a weight whose sides are no multiple of a tile
        dict(name="gemv 37 1537x1440", op="gemv", m=37, n=1537, k=1440, out="bf16"),
        # the norm of one token
        dict(name="ln_fwd 1x4096", op="ln_fwd", rows=1, cols=4096, dtype="bf16"),
        # 64 images x 197 tokens at the MLP width of DeiT-S
        dict(name="ln_fwd 12608x1536", op="ln_fwd", rows=12608, cols=1536, dtype="bf16"),
        # odd sizes in 32 bits
        dict(name="ln_fwd 3001x1111", op="ln_fwd", rows=3001, cols=1111, dtype="f32"),
        # the training step of the same activation
        dict(name="ln_bwd 12608x1536", op="ln_bwd", rows=12608, cols=1536, dtype="bf16"),
        # long rows in 32 bits
        dict(name="ln_bwd 4096x14336", op="ln_bwd", rows=4096, cols=14336, dtype="f32"),
        # a small weight: the products are too short to fill the GPU
        dict(name="ns 256x512", op="ns", rows=256, cols=512, steps=5, dtype="bf16"),
        # an odd, tall weight
        dict(name="ns 1537x1001", op="ns", rows=1537, cols=1001, steps=5, dtype="f32"),
        # an LLM weight
        dict(name="ns 4096x14336", op="ns", rows=4096, cols=14336, steps=5, dtype="bf16"),
    ]


def _log_size(rng, lo, hi, mult=1):
    v = int(round(lo * (hi / lo) ** rng.random()))
    return max(mult, v // mult * mult)


def draw(rng):
    op = rng.choice(["gemv", "ln_fwd", "ln_bwd", "ns"])
    if op == "gemv":
        while True:
            c = dict(op=op, m=_log_size(rng, 1, 64), n=_log_size(rng, 64, 28672),
                     k=_log_size(rng, 256, 28672, rng.choice([32, 128, 128, 128])),
                     out=rng.choice(["bf16", "f32"]))
            if c["n"] * c["k"] <= 8192 * 28672 and c["m"] * c["n"] * c["k"] <= 16 * 4096 * 14336:
                return c
    if op == "ns":
        while True:
            c = dict(op=op, rows=_log_size(rng, 64, 8192), cols=_log_size(rng, 64, 14336),
                     steps=rng.choice([4, 5, 6]), dtype=rng.choice(["bf16", "f32"]))
            if work(c)["flops"] <= 5 * 4096 ** 2 * (3 * 14336 + 4096):
                return c
    while True:
        c = dict(op=op, rows=_log_size(rng, 1, 32768), cols=_log_size(rng, 48, 16384),
                 dtype=rng.choice(["bf16", "f32"]))
        if c["rows"] * c["cols"] <= 4096 * 14336:
            return c


def work(case):
    op = case["op"]
    if op == "gemv":
        m, n, k = case["m"], case["n"], case["k"]
        size = 2 if case["out"] == "bf16" else 4
        return {"bytes": n * k // 2 + n * k // 32 + 2 * m * k + size * m * n, "flops": 2 * m * n * k}
    rows, cols = case["rows"], case["cols"]
    e = rows * cols
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "ln_fwd":
        return {"bytes": 2 * size * e + 8 * cols + 8 * rows, "flops": 8 * e}
    if op == "ln_bwd":
        return {"bytes": 3 * size * e + 12 * cols + 8 * rows, "flops": 14 * e}
    # the Gram matrix and its square are symmetric: half of each is computed
    s, l = min(rows, cols), max(rows, cols)
    return {"bytes": (size + 2) * e, "flops": case["steps"] * (s * s * l + s ** 3 + 2 * s * s * l)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _quantize_rows(w):
    """MXFP4 codes [n, k/2] and scale bytes [n, k/32] of w, nearest value."""
    n, k = w.shape
    g = w.view(n, k // 32, 32)
    amax = g.abs().amax(-1)
    e = (torch.floor(torch.log2(amax.clamp_min(1e-30))) - 2).clamp(-127, 127)
    a = (g.abs() * torch.exp2(-e)[..., None]).view(n, k)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    code = torch.bucketize(a, edges, out_int32=True).to(torch.uint8)
    code = code | ((w < 0).to(torch.uint8) << 3)
    code = code.view(n, k // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).to(torch.uint8)


def _blocked(scales):
    """Scale bytes [n, groups] in the order block-scaled tensor cores read:
    tiles of 128 rows x 4 groups, row r of a tile at 16 (r % 32) + 4 (r // 32)."""
    n, g = scales.shape
    nt, gt = -(-n // 128), -(-g // 4)
    p = torch.zeros((nt * 128, gt * 4), dtype=torch.uint8, device=scales.device)
    p[:n, :g] = scales
    return p.view(nt, 4, 32, gt, 4).permute(0, 3, 2, 1, 4).reshape(nt * 128, gt * 4).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    op = case["op"]
    if op == "gemv":
        m, n, k = case["m"], case["n"], case["k"]
        # activations with a spread of channel sizes and a few outliers
        chan = torch.exp2(4.0 * torch.rand(k, generator=gen, device=DEV) - 2.0)
        chan = torch.where(torch.rand(k, generator=gen, device=DEV) < 0.002, 50.0 * chan, chan)
        x = (normal(m, k) * chan).to(torch.bfloat16)
        codes, scales = _quantize_rows(0.02 * normal(n, k))
        return dict(case, x=x, codes=codes, blocked=_blocked(scales))
    rows, cols = case["rows"], case["cols"]
    dt = DTYPES[case["dtype"]]
    if op == "ns":
        # the momentum of a weight's gradients: a few strong directions and noise
        r = max(1, min(rows, cols) // 16)
        g = normal(rows, r) @ normal(r, cols) / r ** 0.5 + 0.3 * normal(rows, cols)
        return dict(case, g=(1e-3 * g).to(dt))
    chan = torch.exp2(6.6 * torch.rand(cols, generator=gen, device=DEV) - 3.3)
    x = (normal(rows, cols) * chan + 0.3 * normal(cols)).to(dt)
    weight = 1.0 + 0.2 * normal(cols)
    bias = 0.1 * normal(cols)
    if op == "ln_fwd":
        return dict(case, x=x, weight=weight, bias=bias)
    dy = (0.01 * normal(rows, cols)).to(dt)
    xf = x.double() if rows * cols <= 1 << 24 else x.float()
    mean = xf.mean(-1)
    rstd = torch.rsqrt((xf - mean[:, None]).square().mean(-1) + LN_EPS)
    return dict(case, x=x, dy=dy, weight=weight, mean=mean.float(), rstd=rstd.float())


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _decode(codes, blocked, k):
    n = codes.shape[0]
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat([grid, -grid])
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1)
    nt, gt = -(-n // 128), -(-k // 128)
    s = blocked.view(nt, gt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(nt * 128, gt * 4)
    s = torch.exp2(s[:n, : k // 32].float() - 127.0)
    return (v.view(n, k // 32, 32) * s[..., None]).view(n, k)


def _ns_plain(g, steps):
    a, b, c = NS_COEFFS
    x = g.float()
    x = x / (x.square().sum().sqrt() + NS_EPS)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    for _ in range(steps):
        p = x @ x.T
        x = a * x + (b * p + c * (p @ p)) @ x
    return (x.T if tall else x).contiguous().to(torch.bfloat16)


def run(s):
    op = s["op"]
    if own:
        import mxfp4_block_quantization_quantizer_b200 as q
        if op == "gemv":
            return q.gemv(s["x"], s["codes"], s["blocked"], out_dtype=DTYPES[s["out"]])
        if op == "ln_fwd":
            return q.layernorm(s["x"], s["weight"], s["bias"], eps=LN_EPS, want_stats=True)
        if op == "ln_bwd":
            return q.layernorm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
        return q.newton_schulz(s["g"], steps=s["steps"], coeffs=NS_COEFFS, eps=NS_EPS,
                               out_dtype=torch.bfloat16)
    if op == "gemv":
        y = s["x"].float() @ _decode(s["codes"], s["blocked"], s["k"]).T
        return y.to(DTYPES[s["out"]])
    if op == "ln_fwd":
        x = s["x"].float()
        mean = x.mean(-1, keepdim=True)
        d = x - mean
        rstd = 1.0 / (d.square().mean(-1, keepdim=True) + LN_EPS).sqrt()
        y = (d * rstd * s["weight"] + s["bias"]).to(s["x"].dtype)
        return y, mean[:, 0], rstd[:, 0]
    if op == "ln_bwd":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * rstd
        g = dy * s["weight"]
        dx = rstd * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
        return dx.to(s["x"].dtype), (dy * xhat).sum(0), dy.sum(0)
    return _ns_plain(s["g"], s["steps"])


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemv":
        n, k = case["n"], case["k"]
        code = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).reshape(n, k)
        e, f = (code >> 1) & 3, code & 1
        # exponent field 0: 0 or 0.5; else (1 + f / 2) 2^(e - 1)
        mag = torch.where(e == 0, 0.5 * f.double(),
                          (1.0 + 0.5 * f.double()) * torch.exp2(e.double() - 1.0))
        mag = torch.where(code >= 8, -mag, mag)
        r = torch.arange(n, device=DEV)[:, None]
        g = torch.arange(k // 32, device=DEV)[None, :]
        at = ((r // 128) * -(-k // 128) + g // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + g % 4
        scale = torch.exp2(s["blocked"].flatten()[at].double() - 127.0)
        w = mag * scale.repeat_interleave(32, dim=1)
        return s["x"].double() @ w.T
    if op == "ns":
        a, b, c = NS_COEFFS
        x = s["g"].double()
        x = x / (torch.linalg.vector_norm(x) + NS_EPS)
        if x.shape[0] > x.shape[1]:
            for _ in range(case["steps"]):
                p = x.T @ x
                x = a * x + b * (x @ p) + c * ((x @ p) @ p)
        else:
            for _ in range(case["steps"]):
                p = x @ x.T
                x = a * x + b * (p @ x) + c * (p @ (p @ x))
        return x
    x = s["x"].double()
    n = x.shape[1]
    if op == "ln_fwd":
        mean = x.sum(1) / n
        var = ((x - mean[:, None]) ** 2).sum(1) / n
        rstd = (var + LN_EPS) ** -0.5
        y = torch.addcmul(s["bias"].double(), (x - mean[:, None]) * rstd[:, None], s["weight"].double())
        return y, mean, rstd
    mean, rstd = s["mean"].double()[:, None], s["rstd"].double()[:, None]
    h = (x - mean) * rstd
    dy = s["dy"].double()
    dh = dy * s["weight"].double()
    dx = rstd / n * (n * dh - dh.sum(1, keepdim=True) - h * (dh * h).sum(1, keepdim=True))
    return dx, torch.einsum("rc,rc->c", dy, h), torch.einsum("rc->c", dy)
