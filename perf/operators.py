"""Workloads of the operators around the TTT layer in a training step, each in its plain form and as the library's call.

  norm       layer norm of token features, forward and backward (with the gradients of weight and bias)
  rope       rotary positions of Q and K on a token grid (image or video) or at given positions, and its inverse,
             which is its backward pass
  orth       the orthogonal factor of an update by Newton-Schulz products, for weight gradients
  lin_orth   the full-batch TTT-Linear step whose inner update is orthogonalised that way

A case is a dict of plain values; ``prepare`` draws its inputs on the GPU from a seed, ``run`` makes one pass,
``exact`` gives the same outputs from the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
COEF = (3.4445, -4.7750, 2.0315)  # the quintic of the Newton-Schulz step
STEPS = 5
NORM_EPS, ORTH_EPS = 1e-6, 1e-7


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the norm in front of the layer for one 224x224 image at patch 16 with C = 384: latency
        dict(name="norm_fwd_one_image", op="norm", way="fwd", rows=196, cols=384, dtype="bf16", bias=True),
        # a stage-1 batch of 32 images on the 56x56 grid, C = 64: bandwidth, short rows
        dict(name="norm_fwd_stage1", op="norm", way="fwd", rows=32 * 3136, cols=64, dtype="bf16", bias=True),
        # a training batch of 64 images, C = 384
        dict(name="norm_bwd_batch", op="norm", way="bwd", rows=64 * 196, cols=384, dtype="bf16", bias=True),
        # an 80x80 grid and one class token, an odd width, 32-bit training
        dict(name="norm_bwd_odd", op="norm", way="bwd", rows=6401, cols=321, dtype="f32", bias=False),
        # Q and K of one image, 6 heads of 64, straight from the projection's token-major output: latency
        dict(name="rope_one_image", op="rope", B=1, H=6, grid="14x14", dims="32,32", d=64, dtype="bf16",
             tokens=True, given=False, interleaved=False, inverse=False),
        # a video clip, three axes, heads of 128: bandwidth
        dict(name="rope_video", op="rope", B=2, H=12, grid="8x24x24", dims="32,48,48", d=128, dtype="bf16",
             tokens=True, given=False, interleaved=False, inverse=False),
        # gradients of Q and K on the high-resolution grid with a class token, positions given per token
        dict(name="rope_bwd_given", op="rope", B=4, H=3, grid="6401", dims="24,24", d=64, dtype="f32",
             tokens=False, given=True, interleaved=True, inverse=True),
        # the gradients of the heads' inner weights W0
        dict(name="orth_heads", op="orth", U=12, m=64, n=64, dtype="f32"),
        # the gradient of the QKVG projection at C = 384
        dict(name="orth_projection", op="orth", U=1, m=384, n=1536, dtype="f32"),
        # a wide model's projection, 16-bit gradients: arithmetic
        dict(name="orth_wide", op="orth", U=1, m=1024, n=4096, dtype="bf16"),
        # the layer of a small vision transformer, 64 images, 6 heads of 64, 14x14 tokens
        dict(name="lin_orth_batch", op="lin_orth", B=64, H=6, N=196, d=64, dtype="bf16"),
        # the high-resolution stage-1 grid, 56x56 tokens
        dict(name="lin_orth_stage1", op="lin_orth", B=32, H=1, N=3136, d=64, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "rope", "rope", "orth", "orth", "lin_orth"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        cols = _log(rng, 16, 4096)
        if rng.random() < 0.6:
            cols = (cols + 7) // 8 * 8
        rows = _log(rng, 1, min(262144, 12_800_000 // cols))
        return dict(op=op, way=rng.choice(["fwd", "bwd"]), rows=rows, cols=cols, dtype=dtype, bias=rng.random() < 0.7)
    if op == "rope":
        d = rng.choice([32, 64, 64, 96, 128])
        axes = rng.choice([1, 2, 2, 3])
        left = d // 2  # pairs still to share out
        dims = []
        for a in range(axes):
            p = rng.randint(1, left - (axes - 1 - a))
            dims.append(2 * p)
            left -= p
        B, H = _log(rng, 1, 16), rng.choice([1, 2, 3, 6, 12])
        most = 12_000_000 // (B * H * d)
        given = rng.random() < 0.4
        if given:
            N = _log(rng, 1, min(20000, most))
            grid = str(N)
        else:
            side = max(1, int(min(20000, most) ** (1.0 / axes)))
            grid = "x".join(str(rng.randint(1, side)) for _ in range(axes))
        return dict(op=op, B=B, H=H, grid=grid, dims=",".join(map(str, dims)), d=d, dtype=dtype,
                    tokens=rng.random() < 0.5, given=given, interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5)
    if op == "orth":
        if rng.random() < 0.5:  # heads' inner weights
            U, m, n = _log(rng, 1, 64), _log(rng, 8, 128), _log(rng, 8, 256)
        else:  # projections
            U, m = rng.choice([1, 1, 2, 4]), _log(rng, 64, 1024)
            n = _log(rng, 64, 4096)
            while U * min(m, n) ** 2 * max(m, n) > 1024 * 1024 * 4096:
                U = max(1, U // 2)
        if rng.random() < 0.3:
            m, n = n, m
        return dict(op=op, U=U, m=m, n=n, dtype=dtype)
    d = rng.choice([64, 64, 64, 32, 48])
    H = rng.choice([1, 2, 3, 6])
    side = rng.randint(7, 80)
    N = side * rng.randint(max(1, side - 9), side)
    B = _log(rng, 1, max(1, min(64, 6_000_000 // (H * N * d))))
    return dict(op=op, B=B, H=H, N=N, d=d, dtype=dtype)


# ----------------------------------------------------------------------------------- inputs
def _ints(text, sep):
    return [int(t) for t in text.split(sep)]


def _tokens(case):
    return math.prod(_ints(case["grid"], "x"))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "norm":
        rows, cols = case["rows"], case["cols"]
        # features with a spread and an offset of their own, as in a residual stream
        s["x"] = (randn(rows, cols) * (0.5 + randn(cols).abs()) + 0.5 * randn(cols)).to(dt)
        s["gamma"] = 1.0 + 0.2 * randn(cols)
        s["beta"] = 0.2 * randn(cols) if case["bias"] else None
        if case["way"] == "bwd":
            s["dy"] = (0.1 * randn(rows, cols)).to(dt)
    elif case["op"] == "rope":
        B, H, d, N = case["B"], case["H"], case["d"], _tokens(case)
        dims = _ints(case["dims"], ",")
        if case["tokens"]:  # slices of the projection's output, [B, N, 3, H, d]
            qkv = randn(B, N, 3, H, d).to(dt)
            s["q"], s["k"] = qkv[:, :, 0].transpose(1, 2), qkv[:, :, 1].transpose(1, 2)
        else:
            s["q"], s["k"] = randn(B, H, N, d).to(dt), randn(B, H, N, d).to(dt)
        s["dims"], s["grid"], s["pos"] = tuple(dims), None, None
        if case["given"]:  # a longer grid's places, scaled to fractions
            at = torch.rand(N, len(dims), generator=g, device="cuda", dtype=torch.float32)
            s["pos"] = at * 4096.0
            s["pos"][0] = 0.0
        else:
            s["grid"] = tuple(_ints(case["grid"], "x"))
    elif case["op"] == "orth":
        U, m, n = case["U"], case["m"], case["n"]
        r = min(4, m, n)  # gradients: a few strong directions over a bulk
        x = randn(U, m, n) + randn(U, m, r) @ randn(U, r, n)
        s["x"] = (1e-3 * x).to(dt)
    else:
        B, H, N, d = (case[k] for k in ("B", "H", "N", "d"))
        for name in ("q", "k", "v"):
            s[name] = (randn(B, H, N, d) / math.sqrt(d)).to(dt)
        s["w0"] = randn(H, d, d) / math.sqrt(d)
        s["eta"] = 0.2
    return s


# ------------------------------------------------------------------------------ plain forms
def _norm_plain(s):
    x = s["x"].float()
    mean = x.mean(dim=1, keepdim=True)
    xc = x - mean
    rstd = torch.rsqrt((xc * xc).mean(dim=1, keepdim=True) + NORM_EPS)
    xhat = xc * rstd
    if s["case"]["way"] == "fwd":
        y = xhat * s["gamma"]
        return (y if s["beta"] is None else y + s["beta"]).to(s["x"].dtype)
    dy = s["dy"].float()
    t = dy * s["gamma"]
    dx = rstd * (t - t.mean(dim=1, keepdim=True) - xhat * (t * xhat).mean(dim=1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xhat).sum(dim=0),
            "dbeta": dy.sum(dim=0) if s["case"]["bias"] else None}


def _positions(s):
    if s["pos"] is not None:
        return s["pos"].double()
    axes = [torch.arange(n, device=s["q"].device, dtype=torch.float64) for n in s["grid"]]
    return torch.stack([p.reshape(-1) for p in torch.meshgrid(*axes, indexing="ij")], dim=1)


def _rope_plain(s):
    case, d = s["case"], s["case"]["d"]
    pos = _positions(s)
    first, second, angle, at = [], [], [], 0
    for a, width in enumerate(s["dims"]):
        j = torch.arange(width // 2, device=pos.device)
        first.append(at + (2 * j if case["interleaved"] else j))
        second.append(at + (2 * j + 1 if case["interleaved"] else j + width // 2))
        angle.append(pos[:, a, None] * 10000.0 ** (-2.0 * j.double() / width))
        at += width
    first, second, angle = torch.cat(first), torch.cat(second), torch.cat(angle, dim=1)
    cos, sin = angle.cos().float(), angle.sin().float()
    if case["inverse"]:
        sin = -sin
    out = []
    for name in ("q", "k"):
        x = s[name].float()
        y = x.clone(memory_format=torch.contiguous_format)
        x1, x2 = x[..., first], x[..., second]
        y[..., first] = x1 * cos - x2 * sin
        y[..., second] = x2 * cos + x1 * sin
        out.append(y.to(s[name].dtype))
    return out


def _newton_schulz(x):
    """The Newton-Schulz steps in 32 bits, on the side that is shorter."""
    tall = x.shape[-2] > x.shape[-1]
    y = x.float().transpose(-1, -2) if tall else x.float()
    y = y / (y * y).sum(dim=(-2, -1), keepdim=True).sqrt().clamp_min(ORTH_EPS)
    a, b, c = COEF
    for _ in range(STEPS):
        g = y @ y.transpose(-1, -2)
        y = a * y + (b * g + c * (g @ g)) @ y
    return y.transpose(-1, -2) if tall else y


def _lin_orth_plain(s):
    q, k, v, w0 = s["q"].float(), s["k"].float(), s["v"].float(), s["w0"]
    kt = k.transpose(-1, -2)
    grad = (kt @ k @ w0 - kt @ v) / k.shape[2]
    w = w0 - s["eta"] * _newton_schulz(grad)
    return (q @ w).to(s["q"].dtype), w


# ---------------------------------------------------------------------------------- one pass
def run(state):
    s, case = state, state["case"]
    if own:
        from linear_attention_split_b200 import ttt

        if case["op"] == "norm":
            if case["way"] == "fwd":
                return ttt.layernorm(s["x"], s["gamma"], s["beta"], eps=NORM_EPS)
            dx, dgamma, dbeta = ttt.layernorm_bwd(s["dy"], s["x"], s["gamma"], eps=NORM_EPS, with_dbeta=case["bias"])
            return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
        if case["op"] == "rope":
            return list(ttt.rope(s["q"], s["k"], s["dims"], grid=s["grid"], pos=s["pos"],
                                 interleaved=case["interleaved"], inverse=case["inverse"]))
        if case["op"] == "orth":
            return ttt.orthogonalize(s["x"], steps=STEPS, coef=COEF, eps=ORTH_EPS)
        return ttt.linear_fullbatch_orth(s["q"], s["k"], s["v"], s["w0"], eta=s["eta"], steps=STEPS, coef=COEF,
                                         eps=ORTH_EPS, with_w_star=True)
    if case["op"] == "norm":
        return _norm_plain(s)
    if case["op"] == "rope":
        return _rope_plain(s)
    if case["op"] == "orth":
        return _newton_schulz(s["x"]).to(s["x"].dtype)
    return _lin_orth_plain(s)


# -------------------------------------------------------------------------------------- work
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        n, c = case["rows"] * case["cols"], case["cols"]
        if case["way"] == "fwd":
            return {"bytes": 2 * n * es + 4 * c * (2 if case["bias"] else 1), "flops": 8 * n}
        return {"bytes": 3 * n * es + 4 * c * (3 if case["bias"] else 2), "flops": 16 * n}
    if case["op"] == "rope":
        n = 2 * case["B"] * case["H"] * _tokens(case) * case["d"]
        at = 4 * _tokens(case) * len(_ints(case["dims"], ",")) if case["given"] else 0
        return {"bytes": 2 * n * es + at, "flops": 3 * n}

    def steps(m, n):  # symmetric products count once for each pair
        m, n = min(m, n), max(m, n)
        return STEPS * (m * (m + 1) * n + m * (m + 1) * m + 2 * m * m * n)

    if case["op"] == "orth":
        U, m, n = case["U"], case["m"], case["n"]
        return {"bytes": 2 * U * m * n * es, "flops": U * steps(m, n)}
    U, N, d = case["B"] * case["H"], case["N"], case["d"]
    return {"bytes": 4 * U * N * d * es + 4 * (case["H"] + U) * d * d,
            "flops": U * (6 * N * d * d + 2 * d**3 + steps(d, d))}


# --------------------------------------------------------------------------- 64-bit definition
def _orth_exact(x):
    """In the eigenvectors of X X^T every step multiplies the singular value s by a + b s^2 + c s^4."""
    tall = x.shape[-2] > x.shape[-1]
    x = x.transpose(-1, -2) if tall else x
    x = x / torch.linalg.matrix_norm(x).clamp_min(ORTH_EPS)[:, None, None]
    lam, vec = torch.linalg.eigh(x @ x.mT)
    s, gain = lam.clamp_min(0.0).sqrt(), torch.ones_like(lam)
    for _ in range(STEPS):
        p = COEF[0] + COEF[1] * s.square() + COEF[2] * s.pow(4)
        s, gain = s * p, gain * p
    y = (vec * gain[:, None, :]) @ (vec.mT @ x)
    return y.transpose(-1, -2) if tall else y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        x = s["x"].double().requires_grad_()
        gamma = s["gamma"].double().requires_grad_()
        beta = (s["beta"].double() if case["bias"] else torch.zeros_like(gamma)).detach().requires_grad_()
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        y = (x - mean) / (var + NORM_EPS).sqrt() * gamma + beta
        if case["way"] == "fwd":
            return y.detach()
        dx, dgamma, dbeta = torch.autograd.grad(y, (x, gamma, beta), s["dy"].double())
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta if case["bias"] else None}
    if case["op"] == "rope":
        N = _tokens(case)
        pos = s["pos"]
        if pos is None:
            cells, at, stride = torch.arange(N, device="cuda"), [], N
            for size in s["grid"]:
                stride //= size
                at.append(cells // stride % size)
            pos = torch.stack(at, dim=1)
        pos, out = pos.double(), []
        for name in ("q", "k"):
            x, parts = s[name].double(), []
            for a, section in enumerate(torch.split(x, [*s["dims"], case["d"] - sum(s["dims"])], dim=-1)):
                if a == len(s["dims"]):
                    parts.append(section)
                    continue
                half = s["dims"][a] // 2
                shape = (*section.shape[:-1], half, 2) if case["interleaved"] else (*section.shape[:-1], 2, half)
                z = section.reshape(shape) if case["interleaved"] else section.reshape(shape).transpose(-1, -2)
                turn = torch.exp(torch.arange(half, device="cuda").double() * (-math.log(10000.0) / half))
                angle = torch.outer(pos[:, a], turn) * (-1.0 if case["inverse"] else 1.0)
                z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * torch.polar(torch.ones_like(angle), angle))
                parts.append((z if case["interleaved"] else z.transpose(-1, -2)).reshape(section.shape))
            out.append(torch.cat(parts, dim=-1))
        return out
    if case["op"] == "orth":
        return _orth_exact(s["x"].double())
    q, k, v, w0 = s["q"].double(), s["k"].double(), s["v"].double(), s["w0"].double()
    err = k @ w0 - v
    grad = torch.einsum("bhni,bhnj->bhij", k, err) / case["N"]
    B, H, d = case["B"], case["H"], case["d"]
    w = w0 - s["eta"] * _orth_exact(grad.reshape(B * H, d, d)).reshape(B, H, d, d)
    return torch.einsum("bhni,bhij->bhnj", q, w), w
