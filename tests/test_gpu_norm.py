"""Layer norm and its backward pass against the definition in 64 bits (GPU).

Tolerances.  u = 2^-24 is half a step of fp32, h half a step of the output's type (bf16 2^-8, fp32 u).
A row's sums run over at most 16 values in a thread and 10 exchanges, so a mean or a mean square is
within 26 u of the mean of the magnitudes; 32 u leaves room for the mean's own division and the
reciprocal square root.  With m the mean of |t| and of |t xh| below, each output is bounded term by
term:  |dy_out| <= h |y| + 40 u (|xh g| + |g| + |b|)  and
       |d dx| <= h |dx| + 64 u rstd (|t| + m + |xh| m).
The weight sums add rows one after another in a thread (`chain` of them), then over the groups of a
block, then over blocks in 8 strands: (chain + groups + blocks / 8 + 8 + 40) u of the magnitudes' sum,
of which 40 u is the error of xh itself.
"""
import pytest
import torch

from linear_attention_split_b200 import ttt

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
H = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


def draw(rows, C, dt, seed=0, offset=0.0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, C, generator=g) * spread + offset).to(dt)
    dy = torch.randn(rows, C, generator=g).to(dt)
    gamma = 1 + 0.3 * torch.randn(C, generator=g)
    beta = 0.3 * torch.randn(C, generator=g)
    return [t.to(DEV) for t in (x, dy, gamma, beta)]


def stats(x):
    x = x.double()
    c = x - x.mean(-1, keepdim=True)
    rstd = 1 / (c.square().mean(-1, keepdim=True) + EPS).sqrt()
    return c * rstd, rstd


def check_forward(x, gamma, beta, y):
    xh, _ = stats(x)
    g = gamma.double()
    b = torch.zeros_like(g) if beta is None else beta.double()
    want = xh * g + b
    tol = H[x.dtype] * want.abs() + 40 * U * ((xh * g).abs() + g.abs() + b.abs())
    assert ((y.double() - want).abs() <= tol).all(), ((y.double() - want).abs() / tol).max().item()


def check_backward(x, dy, gamma, dx, dgamma, dbeta):
    rows, C = x.shape
    xh, rstd = stats(x)
    d, g = dy.double(), gamma.double()
    t = d * g
    want = rstd * (t - t.mean(-1, keepdim=True) - xh * (t * xh).mean(-1, keepdim=True))
    m = t.abs().mean(-1, keepdim=True) + (t * xh).abs().mean(-1, keepdim=True)
    tol = H[x.dtype] * want.abs() + 64 * U * rstd * (t.abs() + m + xh.abs() * m)
    assert ((dx.double() - want).abs() <= tol).all(), ((dx.double() - want).abs() / tol).max().item()
    # at least 148 blocks' worth of strands unless there are few rows: `chain` of the fewest blocks
    chain = rows / 148 + 1
    adds = chain + 256 + 2 * 148 / 8 + 8 + 40
    for got, terms in ((dgamma, d * xh), (dbeta, d)):
        if got is None:
            continue
        tol = adds * U * (terms.abs().sum(0) + (d.abs().sum(0) if got is dgamma else 0))
        diff = (got.double() - terms.sum(0)).abs()
        assert (diff <= tol).all(), (diff / tol).max().item()


SHAPES = [(1, 1), (1, 2), (3, 5), (7, 8), (2, 31), (5, 33), (196, 64), (197, 96), (50, 100), (33, 257), (6401, 321),
          (300, 384), (64, 768), (19, 1000), (9, 1024), (5, 2056), (4, 4097), (3, 8192), (2, 16384), (2, 16383), (40000, 16)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C", SHAPES)
def test_norm_forward_and_backward(rows, C, dtype):
    x, dy, gamma, beta = draw(rows, C, DT[dtype], seed=rows + C)
    check_forward(x, gamma, beta, ttt.layernorm(x, gamma, beta, EPS))
    check_forward(x, gamma, None, ttt.layernorm(x, gamma, None, EPS))
    check_backward(x, dy, gamma, *ttt.layernorm_bwd(dy, x, gamma, EPS))
    dx, dgamma, none = ttt.layernorm_bwd(dy, x, gamma, EPS, with_dbeta=False)
    assert none is None
    check_backward(x, dy, gamma, dx, dgamma, None)
    assert ttt.device_error() == 0


@pytest.mark.parametrize("offset,spread", [(1e4, 1.0), (-300.0, 1e-2), (0.0, 1e-4), (0.0, 1e8), (1e6, 3.0)])
def test_norm_of_rows_far_from_zero(offset, spread):
    # the stored values are what counts: x - mean is exact to u |offset| before the second mean takes out
    # the rest, so the bound is the one above
    x, dy, gamma, beta = draw(65, 320, torch.float32, seed=3, offset=offset, spread=spread)
    check_forward(x, gamma, beta, ttt.layernorm(x, gamma, beta, EPS))
    check_backward(x, dy, gamma, *ttt.layernorm_bwd(dy, x, gamma, EPS))


def test_norm_of_constant_rows_is_the_bias():
    x = torch.full((6, 48), 3.25, device=DEV)
    _, dy, gamma, beta = draw(6, 48, torch.float32)
    assert torch.equal(ttt.layernorm(x, gamma, beta, EPS), beta.expand(6, 48))
    dx, dgamma, dbeta = ttt.layernorm_bwd(dy, x, gamma, EPS)
    assert (dgamma == 0).all() and torch.isfinite(dx).all()


def test_norm_with_an_outlier_feature():
    x, dy, gamma, beta = draw(70, 384, torch.float32, seed=9)
    x[:, 0] = 1e5
    check_forward(x, gamma, beta, ttt.layernorm(x, gamma, beta, EPS))
    check_backward(x, dy, gamma, *ttt.layernorm_bwd(dy, x, gamma, EPS))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("C", [24, 321, 2048])
def test_norm_nonfinite_stays_in_its_row(bad, C):
    x, dy, gamma, beta = draw(20, C, torch.bfloat16, seed=1)
    clean = ttt.layernorm(x, gamma, beta, EPS)
    cdx = ttt.layernorm_bwd(dy, x, gamma, EPS)[0]
    x[7, C // 2] = bad
    y = ttt.layernorm(x, gamma, beta, EPS)
    dx = ttt.layernorm_bwd(dy, x, gamma, EPS)[0]
    rest = [i for i in range(20) if i != 7]
    assert torch.equal(y[rest], clean[rest]) and torch.equal(dx[rest], cdx[rest])
    assert y[7].isnan().all() and dx[7].isnan().all()


def test_norm_shapes_in_place_and_strides():
    x, dy, gamma, beta = draw(60, 64, torch.bfloat16)
    want = ttt.layernorm(x, gamma, beta, EPS)
    assert torch.equal(ttt.layernorm(x.view(3, 4, 5, 64), gamma, beta, EPS), want.view(3, 4, 5, 64))
    grads = ttt.layernorm_bwd(dy, x, gamma, EPS)
    for target in ("dy", "x"):
        a, b = dy.clone(), x.clone()
        dx = a if target == "dy" else b
        dgamma, dbeta = torch.empty_like(gamma), torch.empty_like(gamma)
        ttt.ttt_layernorm_bwd(a, b, gamma, dx, dgamma, dbeta, EPS)
        for got, ref in zip((dx, dgamma, dbeta), grads):
            assert torch.equal(got, ref)
    y = x.clone()
    ttt.ttt_layernorm(y, gamma, beta, y, EPS)
    assert torch.equal(y, want)
    with pytest.raises(ValueError):
        ttt.layernorm(x[:, ::2], gamma[:32], None)
    with pytest.raises(ValueError):
        ttt.layernorm(x, gamma[:32], None)
    with pytest.raises(ValueError):
        ttt.ttt_layernorm(x, gamma, beta, torch.empty_like(x)[:59])


@pytest.mark.parametrize("rows,C,dtype", [(12544, 384, "bf16"), (6401, 321, "f32"), (3, 5000, "bf16")])
def test_norm_is_deterministic(rows, C, dtype):
    x, dy, gamma, beta = draw(rows, C, DT[dtype])
    a, b = ttt.layernorm_bwd(dy, x, gamma, EPS), ttt.layernorm_bwd(dy, x, gamma, EPS)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_norm_gradient_by_differences():
    # central differences of a 64-bit loss through the fp32 forward's definition, at scattered places
    x, dy, gamma, beta = draw(4, 37, torch.float32, seed=5)
    dx, dgamma, dbeta = ttt.layernorm_bwd(dy, x, gamma, EPS)

    def loss(x, g, b):
        xh, _ = stats(x)
        return ((xh * g + b) * dy.double()).sum().item()

    args = [x.double(), gamma.double(), beta.double()]
    for i, got in enumerate((dx, dgamma, dbeta)):
        for e in range(0, got.numel(), 11):
            ends = []
            for s in (1e-5, -1e-5):
                moved = [a.clone() for a in args]
                moved[i].view(-1)[e] += s
                ends.append(loss(*moved))
            # step^2 third derivative and the loss' own rounding: both below 1e-6 here
            assert abs((ends[0] - ends[1]) / 2e-5 - got.view(-1)[e].item()) < 2e-5 * max(1.0, dy.abs().sum().item())


def test_norm_guard_bands():
    for rows, C, dt in ((7, 321, torch.bfloat16), (33, 96, torch.float32), (5, 2056, torch.bfloat16)):
        x, dy, gamma, beta = draw(rows, C, dt)
        margin = 4096
        nb = ttt.ttt_layernorm_bwd_workspace_bytes(rows, C, ttt._DT[dt])

        def guarded(n, dtype):
            es = torch.empty((), dtype=dtype).element_size()
            raw = torch.full((2 * margin + n * es,), 0xA5, dtype=torch.uint8, device=DEV)
            return raw, raw[margin:margin + n * es].view(dtype)

        raws = {}
        for name, n, d in (("y", rows * C, dt), ("dx", rows * C, dt), ("dg", C, torch.float32), ("db", C, torch.float32),
                           ("ws", nb, torch.uint8)):
            raws[name] = guarded(n, d)
        ttt.ttt_layernorm(x, gamma, beta, raws["y"][1].view(rows, C), EPS)
        ttt.ttt_layernorm_bwd(dy, x, gamma, raws["dx"][1].view(rows, C), raws["dg"][1], raws["db"][1], EPS, raws["ws"][1])
        torch.cuda.synchronize()
        for raw, t in raws.values():
            n = t.numel() * t.element_size()
            assert (raw[:margin] == 0xA5).all() and (raw[margin + n:] == 0xA5).all()
        check_forward(x, gamma, beta, raws["y"][1].view(rows, C))


def test_norm_past_32_bit_offsets():
    # 2^31 elements and a few rows: the last rows lie behind what a 32-bit element offset reaches
    rows, C = 524288 + 37, 4096
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of free device memory")
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.empty(rows, C, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    gamma = 1 + 0.1 * torch.randn(C, generator=g, device=DEV)
    y = ttt.layernorm(x, gamma, None, EPS)
    ends = [0, 1, 524287, 524288, rows - 1]
    check_forward(x[ends], gamma, None, y[ends])
    # x as its own gradient: dx of those rows, and the weight's sum over all of them against torch in 64 bits by pieces
    dx, dgamma, _ = ttt.layernorm_bwd(x, x, gamma, EPS, with_dbeta=False)
    small = ttt.layernorm_bwd(x[ends].contiguous(), x[ends].contiguous(), gamma, EPS)[0]
    assert torch.equal(dx[ends], small)
    want, size = torch.zeros(C, dtype=torch.float64, device=DEV), torch.zeros(C, dtype=torch.float64, device=DEV)
    for i in range(0, rows, 32768):
        terms = x[i:i + 32768].double() * stats(x[i:i + 32768])[0]
        want += terms.sum(0)
        size += terms.abs().sum(0) + x[i:i + 32768].double().abs().sum(0)
    adds = rows / 148 + 256 + 2 * 148 / 8 + 8 + 40  # as above: `chain` of the fewest blocks
    assert ((dgamma.double() - want).abs() <= adds * U * size).all()
