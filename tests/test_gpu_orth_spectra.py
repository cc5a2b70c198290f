"""Newton-Schulz steps of matrices with one strong direction, in 64 bits (GPU).

Where one singular value outweighs the rest, the others start near 0 and every step enlarges them, and
whatever rounding has put beside them, by up to a = 3.4445: a^5 = 485 over five steps.  The bounds below
hold for any spectrum.

A bf16 result is rounded by 2^-8 / sqrt(3) = 2.3e-3 of its norm at most, on average over its values (2^-8 for
each).  X and P of the last step are held in 11 bits, 2^-11 / sqrt(3) = 2.8e-4 of X's norm times the polynomial's
largest slope (3.97 on [0, 1.2024], where the values lie then) and times its largest a + b s^2 + c s^4 (3.4445);
the result's norm is at least 0.639 of X's, the least a + b s^2 + c s^4 there: 1.75e-3 and 1.52e-3.  What the
steps before leave is 5 a^5 2^-22 = 5.8e-4 at most (operands of 22 bits), 1.2e-3 of a result of norm 1/2 or
more.  The root of the squares is 3.5e-3, inside 2^-8 = 3.9e-3.
"""
import pytest
import torch

from linear_attention_split_b200 import ttt

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def steps64(x, steps=5, coef=ttt.NS_COEF):
    x = x.double()
    x = x.mT if x.shape[-2] > x.shape[-1] else x
    x = x / torch.linalg.matrix_norm(x)[..., None, None]
    a, b, c = coef
    for _ in range(steps):
        g = x @ x.mT
        x = a * x + (b * g + c * g @ g) @ x
    return x


def draw(kind, weight, U, m, n, dt):
    g = torch.Generator().manual_seed(m + n + weight)
    x = torch.randn(U, m, n, generator=g)
    if kind == "direction":
        x += weight * torch.randn(U, m, 1, generator=g) @ torch.randn(U, 1, n, generator=g)
    elif kind == "offset":
        x += weight
    elif kind == "few rows":  # the strong direction lies in four rows
        x[:, :4] += weight * torch.randn(U, 4, 1, generator=g) @ torch.randn(U, 1, n, generator=g)
    return (1e-3 * x).to(dt).to(DEV)


def error(x, got, **kw):
    want = steps64(x, **kw)
    got = got.double().mT if x.shape[-2] > x.shape[-1] else got.double()
    size = torch.linalg.matrix_norm(want)
    assert (size >= 0.5).all()
    return (torch.linalg.matrix_norm(got - want) / size).max().item()


KINDS = [("direction", 10), ("direction", 30), ("direction", 100), ("direction", 1000), ("offset", 30), ("offset", 1000),
         ("few rows", 300)]
SHAPES = [(1, 256, 512), (2, 72, 300), (1, 1000, 300), (1, 65, 64), (3, 128, 128), (1, 1024, 1024), (2, 64, 256), (1, 200, 4096)]


@pytest.mark.parametrize("U,m,n", SHAPES)
@pytest.mark.parametrize("kind,weight", KINDS)
def test_bf16_with_a_strong_direction(kind, weight, U, m, n):
    x = draw(kind, weight, U, m, n, torch.bfloat16)
    assert error(x, ttt.orthogonalize(x)) <= 2.0 ** -8
    assert ttt.device_error() == 0


# one step of a steep polynomial (slope 5 at 0), eight of the usual one, six of one that flattens at 1
# (slopes of the last two steps: 2 in all).  One step of (5, -6, 2): everything but the result's rounding is 22 bits;
# more steps: the bound of the head, with smaller gains for (2, -1.5, 0.5) (2^6 = 64, slope 2 twice)
@pytest.mark.parametrize("steps,coef", [(1, (5.0, -6.0, 2.0)), (1, ttt.NS_COEF), (2, ttt.NS_COEF), (6, (2.0, -1.5, 0.5))])
@pytest.mark.parametrize("m,n", [(96, 400), (300, 130)])
def test_bf16_other_steps(steps, coef, m, n):
    x = draw("direction", 20, 2, m, n, torch.bfloat16)
    assert error(x, ttt.orthogonalize(x, steps=steps, coef=coef), steps=steps, coef=coef) <= 2.0 ** -8


@pytest.mark.parametrize("U,m,n", SHAPES + [(12, 64, 64), (1, 384, 1536)])
@pytest.mark.parametrize("kind,weight", [("direction", 1)] + KINDS)
def test_f32_with_a_strong_direction(kind, weight, U, m, n):
    # every step leaves 2^-22 of its norm, which the steps after it enlarge by 3.4445 each at most
    x = draw(kind, weight, U, m, n, torch.float32)
    size = torch.linalg.matrix_norm(steps64(x)).min().item()
    assert error(x, ttt.orthogonalize(x)) <= 5 * 3.4445 ** 5 * 2.0 ** -22 / size


# One step of (0, 1, 0) is (X X^T) X, two long sums.  The tensor cores cut every addition to 24 bits of what has
# been summed so far (2^-23 of it at most): n additions into one accumulator that grows evenly lose n / 2 of these.
# An accumulator takes 50 at most (four for 64 terms).  X, A and P are stored to 2^-22.  256 additions into one
# accumulator would lose 1.5e-5 at most and half of that on average.
@pytest.mark.parametrize("U,m,n", [(1, 1024, 4096), (1, 384, 1536), (1, 128, 20000), (24, 100, 5000), (2, 1500, 1500), (1, 4096, 512)])
def test_f32_long_sums(U, m, n):
    g = torch.Generator().manual_seed(m + n)
    x = torch.randn(U, m, n, generator=g).to(DEV)
    x = x / torch.linalg.matrix_norm(x)[..., None, None]
    got = ttt.orthogonalize(x, steps=1, coef=(0.0, 1.0, 0.0)).double()
    d = x.double()
    want = d @ (d.mT @ d) if m > n else (d @ d.mT) @ d
    adds = sum(min(50, 4 * ((k + 63) // 64)) for k in (m, n))
    off = torch.linalg.matrix_norm(got - want) / torch.linalg.matrix_norm(want)
    assert (off <= adds / 2 * 2.0 ** -23 + 3 * 2.0 ** -22).all(), off.max().item()


# What include/ttt.h promises of fp32 matrices without a strong direction after five steps of the usual quintic: 5e-6 of
# the norm.  (1e-6 to 3.6e-6 here.  With one accumulator for a product's hi hi terms 1024 x 4096 is 1.3e-5 off, 384 x 1536
# 6e-6; with the K blocks in ascending order 4 x 1024 x 1024 8e-6, 2048 x 2048 1.5e-5 and 2048 x 8192 2.2e-5.)
@pytest.mark.parametrize("U,m,n", [(1, 1024, 4096), (1, 384, 1536), (1, 1024, 1024), (1, 200, 4096), (1, 128, 20000), (1, 300, 72),
                                   (24, 100, 5000), (12, 64, 64), (8, 1024, 1024), (64, 256, 2048), (1, 1500, 1500), (1, 1500, 4096),
                                   (1, 2048, 2048), (1, 8192, 2048), (1, 4096, 4096), (4, 1024, 1024), (64, 512, 512), (2, 900, 1000)])
def test_f32_of_random_matrices_is_as_good_as_promised(U, m, n):
    g = torch.Generator(device=DEV).manual_seed(m + n)
    x = torch.randn(U, m, n, generator=g, device=DEV)
    x += torch.randn(U, m, 1, generator=g, device=DEV) @ torch.randn(U, 1, n, generator=g, device=DEV)
    assert error(x, ttt.orthogonalize(x)) <= 5e-6


# Small fp32 matrices, the error of 24 of them together.  A step stores X, A and P to 22 bits, 2^-22 / sqrt(3) = 1.4e-7 of
# their norms each, sqrt(3) x 1.4e-7 = 2.4e-7 for a step, and gains of about 2 over the steps that follow for these
# spectra: sqrt(5) x 2 x 2.4e-7 = 1.1e-6; cut additions of X X^T add 2^-24 for each of up to 16, in its share of the step:
# 1e-6 for 256 columns.  With a in P's diagonal, where the accumulator cuts all of a X, 33 x 64 is 2.5e-6 off, 45 x 81 2.6e-6,
# 64 x 200 3.4e-6 and 64 x 256 3.7e-6.
@pytest.mark.parametrize("rank", [0, 3])
@pytest.mark.parametrize("m,n,tol", [(64, 64, 2e-6), (33, 64, 2e-6), (17, 33, 2e-6), (45, 81, 2e-6), (81, 45, 2e-6), (64, 200, 3e-6), (64, 256, 3e-6),
                                     (256, 64, 3e-6), (8, 8, 2e-6), (5, 7, 2e-6), (12, 100, 2e-6), (1, 9, 2e-6)])
def test_f32_small_matrices(m, n, tol, rank):
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(24, m, n, generator=g, device=DEV)
    if rank:
        x += torch.randn(24, m, rank, generator=g, device=DEV) @ torch.randn(24, rank, n, generator=g, device=DEV)
    want, got = steps64(x), ttt.orthogonalize(x).double()
    got = got.mT if m > n else got
    assert (got - want).norm() <= tol * want.norm()
