"""Newton-Schulz orthogonalisation, and the TTT-Linear step that uses it, in 64 bits (GPU).

Tolerance of the iteration.  Every step rounds its products to about d = 2^-22 of their norm (fp32 sums
of operands held to 22 bits or more), and a step enlarges what is already wrong by at most a = 3.4445.
With |X_0| = 1 five steps leave at most 5 a^5 d = 5.8e-4 in the Frobenius norm in the worst direction, and
the result has norm about sqrt(r), r the rank: TOL / sqrt(r) of it.  A bf16 result may be half a step,
2^-8, of each value off.  Rounding takes 2^-8 / sqrt(3) of that on average (2.3e-3 at most, values being
spread over their binades 1.7e-3); X and P of bf16 matrices are held in 11 bits, 2^-11 / sqrt(3) = 2.8e-4
of the norm each at each of five steps: 5 x 2 x 2.8e-4 = 2.8e-3 if all added up, sqrt(10) x 2.8e-4 = 0.9e-3
as independent errors.  The root of the squares, 2.5e-3 at the most, is inside 2^-8 = 3.9e-3.
"""
import math

import pytest
import torch

import oracle
from linear_attention_split_b200 import inputs, ttt
from tolerance import assert_close

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = 5 * 3.4445 ** 5 * 2.0 ** -22


def steps64(x, steps=5, coef=ttt.NS_COEF, eps=1e-7):
    x = x.double()
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    x = x / torch.linalg.matrix_norm(x).clamp_min(eps)[..., None, None]
    a, b, c = coef
    for _ in range(steps):
        g = x @ x.mT
        x = a * x + (b * g + c * g @ g) @ x
    return x.mT if tall else x


def draw(U, m, n, dt, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = min(3, m, n)
    x = torch.randn(U, m, n, generator=g) + torch.randn(U, m, r, generator=g) @ torch.randn(U, r, n, generator=g)
    return (1e-3 * x).to(dt).to(DEV)


def check(got, x, **kw):
    scale = kw.pop("scale", 1.0)
    want = steps64(x, **kw) * scale
    off = torch.linalg.matrix_norm(got.double() - want)
    size = torch.linalg.matrix_norm(want)
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    assert (off <= half * size + TOL * abs(scale)).all(), (off / size).max().item()


SHAPES = [(1, 1, 1), (3, 1, 7), (2, 7, 1), (5, 3, 4), (2, 16, 16), (7, 17, 33), (12, 64, 64), (3, 64, 256), (2, 256, 64), (2, 63, 65),
          (4, 65, 64), (2, 128, 128), (3, 100, 130), (1, 129, 200), (2, 320, 320), (1, 384, 1536), (1, 1000, 72), (1, 513, 520),
          (65, 32, 32), (1, 64, 4096), (1, 1024, 1024), (1, 1, 5000), (2, 3, 1000), (1, 5000, 3), (200, 70, 72), (3, 576, 600),
          (450, 33, 64), (1, 2048, 192)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("U,m,n", SHAPES)
def test_orthogonalize(U, m, n, dtype):
    x = draw(U, m, n, DT[dtype], seed=m + n)
    before = x.clone()
    check(ttt.orthogonalize(x), x)
    assert torch.equal(x, before)
    assert ttt.device_error() == 0


@pytest.mark.parametrize("shape", [(2, 40, 24), (1, 130, 140)])
def test_orthogonalize_arguments(shape):
    x = draw(*shape, torch.float32)
    for steps in (1, 2, 8):
        check(ttt.orthogonalize(x, steps=steps, scale=-0.25), x, steps=steps, scale=-0.25)
    check(ttt.orthogonalize(x, coef=(2.0, -1.5, 0.5), steps=6), x, coef=(2.0, -1.5, 0.5), steps=6)
    check(ttt.orthogonalize(x, eps=10.0), x, eps=10.0)  # a floor above the norm
    out = torch.empty_like(x)
    assert ttt.ttt_orthogonalize(x, out) is out
    want = out.clone()
    y = x.clone()
    ttt.ttt_orthogonalize(y, y)  # in place
    assert torch.equal(y, want)
    assert torch.equal(ttt.orthogonalize(x[0]), want[0])  # one matrix, [m, n]


@pytest.mark.parametrize("m,n", [(24, 40), (64, 64), (130, 70), (300, 200)])
@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e12, 1e30])
def test_orthogonalize_of_any_size_of_values(m, n, scale):
    x = draw(1, m, n, torch.float32) * (1e3 * scale)
    check(ttt.orthogonalize(x, eps=1e-37), x, eps=1e-37)


@pytest.mark.parametrize("m,n", [(16, 16), (64, 64), (64, 200), (96, 130), (256, 256)])
def test_orthogonalize_special_matrices(m, n):
    z = torch.zeros(3, m, n, device=DEV)
    assert (ttt.orthogonalize(z) == 0).all()
    x = draw(4, m, n, torch.float32)
    clean = ttt.orthogonalize(x)
    x[1, 0, 0], x[2] = float("nan"), 0.0
    x[3, m - 1, n - 1] = float("inf")
    got = ttt.orthogonalize(x)
    assert torch.equal(got[0], clean[0])  # its neighbours change nothing
    assert got[1].isnan().all() and got[3].isnan().all() and (got[2] == 0).all()
    # rank one: the one singular value goes through the polynomial alone
    u, v = torch.randn(m, 1, generator=torch.Generator().manual_seed(1)).to(DEV), torch.ones(1, n, device=DEV)
    check(ttt.orthogonalize((u @ v)[None]), (u @ v)[None])
    # an orthogonal factor already: all singular values equal
    q = torch.linalg.qr(draw(1, n, m, torch.float32) if n >= m else draw(1, m, n, torch.float32))[0].mT.contiguous()
    check(ttt.orthogonalize(q), q)


@pytest.mark.parametrize("U,m,n,dtype", [(12, 64, 64, "f32"), (1, 384, 1536, "f32"), (1, 512, 640, "bf16")])
def test_orthogonalize_is_deterministic(U, m, n, dtype):
    x = draw(U, m, n, DT[dtype])
    assert torch.equal(ttt.orthogonalize(x), ttt.orthogonalize(x))


def test_orthogonalize_matrices_do_not_depend_on_their_batch():
    x = draw(9, 64, 64, torch.float32)
    got = ttt.orthogonalize(x)
    for u in (0, 4, 8):
        assert torch.equal(ttt.orthogonalize(x[u]), got[u])


@pytest.mark.parametrize("U,m,n,dt", [(3, 17, 33, torch.float32), (2, 64, 64, torch.bfloat16), (1, 130, 257, torch.bfloat16),
                                      (1, 257, 130, torch.float32)])
def test_orthogonalize_guard_bands(U, m, n, dt):
    x = draw(U, m, n, dt)
    margin, es = 65536, x.element_size()
    nb = ttt.ttt_orthogonalize_workspace_bytes(U, m, n, ttt._DT[dt])
    out = torch.full((2 * margin + U * m * n * es,), 0xA5, dtype=torch.uint8, device=DEV)
    ws = torch.full((2 * margin + nb,), 0xA5, dtype=torch.uint8, device=DEV)
    o = out[margin:margin + U * m * n * es].view(dt).view(U, m, n)
    for _ in range(2):  # a used workspace as well as a fresh one
        ttt.ttt_orthogonalize(x, o, workspace=ws[margin:margin + nb])
        torch.cuda.synchronize()
        for raw, n_in in ((out, U * m * n * es), (ws, nb)):
            assert (raw[:margin] == 0xA5).all() and (raw[margin + n_in:] == 0xA5).all()
        check(o, x)


# ---------------------------------------------------------------- the TTT-Linear step with it
def linear_orth64(inp, eta, steps=5):
    q, k, v, w0 = (inp[n].double() for n in ("q", "k", "v", "w0"))
    grad = (k.mT @ (k @ w0 - v)) / k.shape[2]
    w = w0 - eta * steps64(grad, steps)
    return q @ w, w


LINEAR = [(1, 1, 196, 64, "bf16"), (2, 3, 197, 64, "bf16"), (64, 2, 49, 64, "bf16"), (3, 1, 3136, 64, "bf16"), (1, 2, 1000, 32, "bf16"),
          (2, 2, 100, 48, "bf16"), (1, 2, 196, 64, "f32"), (2, 2, 333, 32, "f32"), (1, 1, 77, 128, "f32"), (1, 1, 50, 5, "f32"),
          (5, 3, 640, 64, "f32"), (1, 1, 128, 128, "bf16"), (1, 1, 64, 1, "f32"),
          (2, 2, 100, 8, "bf16"), (3, 2, 130, 40, "bf16"), (2, 1, 65, 56, "bf16"), (2, 2, 90, 20, "bf16"), (150, 2, 60, 32, "bf16"),
          (1, 2, 200, 96, "f32"), (2, 1, 333, 70, "f32"), (2, 2, 65, 33, "f32")]


@pytest.mark.parametrize("B,H,N,d,dtype", LINEAR)
def test_linear_orth(B, H, N, d, dtype):
    inp = inputs.linear_inputs(B, H, N, d, dtype=dtype, seed=N + d)
    g = {k: v.to(DEV) for k, v in inp.items()}
    out, ws = ttt.linear_fullbatch_orth(g["q"], g["k"], g["v"], g["w0"], eta=0.2, with_w_star=True)
    ro, rw = linear_orth64(inp, 0.2)
    assert_close(out, ro.numpy(), DT[dtype], "orth O")
    assert_close(ws, rw.numpy(), torch.float32, "orth W*")  # W* is fp32 for either input type
    assert torch.equal(ttt.linear_fullbatch_orth(g["q"], g["k"], g["v"], g["w0"], eta=0.2), out)
    assert ttt.device_error() == 0


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 32), ("f32", 64)])
def test_linear_orth_special_cases(dtype, d):
    inp = inputs.linear_inputs(2, 2, 130, d, dtype=dtype, seed=4)
    g = {k: v.to(DEV) for k, v in inp.items()}
    # eta = 0: the forward pass of W0 (the oracle's full-batch step at eta = 0)
    out, ws = ttt.linear_fullbatch_orth(g["q"], g["k"], g["v"], g["w0"], eta=0.0, with_w_star=True)
    assert torch.equal(ws, g["w0"].expand(2, 2, d, d))
    assert_close(out, oracle.linear_fullbatch(inp["q"], inp["k"], inp["v"], inp["w0"], eta=0.0)[0], DT[dtype], "eta 0")
    # no tokens that say anything: K = 0 has no gradient
    zero = torch.zeros_like(g["k"])
    _, ws = ttt.linear_fullbatch_orth(g["q"], zero, g["v"], g["w0"], eta=0.3, with_w_star=True)
    assert torch.equal(ws, g["w0"].expand(2, 2, d, d))
    # one token: the gradient has rank one
    one = {n: t[:, :, :1].contiguous() if n != "w0" else t for n, t in inp.items()}
    o1 = {k: v.to(DEV) for k, v in one.items()}
    out, ws = ttt.linear_fullbatch_orth(o1["q"], o1["k"], o1["v"], o1["w0"], eta=0.2, with_w_star=True)
    ro, rw = linear_orth64(one, 0.2)
    assert_close(out, ro.numpy(), DT[dtype], "one token O")
    assert_close(ws, rw.numpy(), torch.float32, "one token W*")


@pytest.mark.parametrize("dtype,N,d", [("bf16", 3136, 64), ("f32", 700, 64), ("bf16", 333, 48), ("bf16", 130, 24), ("f32", 99, 33)])
def test_linear_orth_is_deterministic_and_in_bounds(dtype, N, d):
    inp = inputs.linear_inputs(2, 3, N, d, dtype=dtype, seed=8)
    g = {k: v.to(DEV) for k, v in inp.items()}
    want = ttt.linear_fullbatch_orth(g["q"], g["k"], g["v"], g["w0"], eta=0.2)
    margin, nbytes = 65536, g["q"].numel() * g["q"].element_size()
    nb = ttt.ttt_linear_fullbatch_orth_workspace_bytes(2, 3, N, d, ttt._DT[g["q"].dtype])
    raw = torch.full((2 * margin + nbytes,), 0xA5, dtype=torch.uint8, device=DEV)
    ws = torch.full((2 * margin + nb,), 0xA5, dtype=torch.uint8, device=DEV)
    out = raw[margin:margin + nbytes].view(g["q"].dtype).view(g["q"].shape)
    ttt.ttt_linear_fullbatch_orth(g["q"], g["k"], g["v"], g["w0"], out, eta=0.2, workspace=ws[margin:margin + nb])
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    for r, n in ((raw, nbytes), (ws, nb)):
        assert (r[:margin] == 0xA5).all() and (r[margin + n:] == 0xA5).all()


def test_math_is_sane():
    # the bound of the file's head is what its comment says
    assert math.isclose(TOL, 5.78e-4, rel_tol=0.01)
