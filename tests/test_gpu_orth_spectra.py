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
