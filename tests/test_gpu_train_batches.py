"""Many matrices or units in one call (GPU): more than two for each SM, where the one-block kernels are compiled for
three blocks an SM, and long units whose tokens are not split.

A matrix of at most 64 x 256 takes the same operations in the same order whatever its batch, so its result is the
same bit for bit.  A larger one may be cut into other tiles in another batch, and a unit's tokens into other splits:
those are held to the bound of their operator each time.
"""
import pytest
import torch

from linear_attention_split_b200 import ttt
from test_gpu_orth import check, steps64
from test_gpu_orth_spectra import error
from tolerance import assert_close

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,n", [(64, 64), (33, 200), (200, 64), (5, 7), (64, 256)])
def test_small_matrices_by_themselves_and_among_many(m, n, dtype):
    few = 2 * torch.cuda.get_device_properties(0).multi_processor_count  # the most for two blocks an SM
    x = randn(few + 150, m, n, seed=m + n).to(DT[dtype])
    got = ttt.orthogonalize(x)
    check(got, x)
    assert torch.equal(ttt.orthogonalize(x[:few + 1]), got[:few + 1])
    assert torch.equal(ttt.orthogonalize(x[:few]), got[:few])
    for u in (0, few - 1, few, few + 149):
        assert torch.equal(ttt.orthogonalize(x[u:u + 1].clone())[0], got[u])


@pytest.mark.parametrize("dtype,tol", [("f32", 5e-6), ("bf16", 2.0 ** -8)])
@pytest.mark.parametrize("m,n", [(130, 257), (384, 512), (257, 64)])
def test_large_matrices_by_themselves_and_among_many(m, n, dtype, tol):
    x = randn(40, m, n, seed=m + n).to(DT[dtype])
    for U in (1, 2, 4, 9, 40):
        assert error(x[:U], ttt.orthogonalize(x[:U])) <= tol


def linear64(q, k, v, w0, eta):
    k64 = k.double()
    w = w0.double() - eta * steps64((k64.mT @ (k64 @ w0.double() - v.double())) / k.shape[2])
    return q.double() @ w, w


def units(q, k, v, w0, out, w, B, H, eta=0.2):
    for b, h in {(0, 0), (0, H - 1), (B // 2, H // 2), (B - 1, 0), (B - 1, H - 1)}:
        one = [t[b:b + 1, h:h + 1] for t in (q, k, v)]
        ro, rw = linear64(*one, w0[h:h + 1], eta)
        assert_close(out[b:b + 1, h:h + 1], ro.cpu().numpy(), out.dtype, f"O {b} {h}")
        assert_close(w[b:b + 1, h:h + 1], rw.cpu().numpy(), torch.float32, f"W* {b} {h}")


# a unit per block, two and three blocks an SM on either side of 296 units; whole and padded heads; a single token
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,N,d", [(148, 2, 60, 64), (150, 2, 60, 64), (64, 6, 196, 64), (445, 1, 33, 64), (1000, 1, 1, 64), (150, 2, 60, 48),
                                     (297, 1, 50, 30)])
def test_linear_orth_of_many_units(B, H, N, d, dtype):
    q, k, v = (randn(B, H, N, d, seed=s).div(d ** 0.5).to(DT[dtype]) for s in (1, 2, 3))
    w0 = randn(H, d, d, seed=4) / d ** 0.5
    out, w = ttt.linear_fullbatch_orth(q, k, v, w0, eta=0.2, with_w_star=True)
    units(q, k, v, w0, out, w, B, H)
    assert torch.equal(ttt.linear_fullbatch_orth(q, k, v, w0, eta=0.2), out)
    assert ttt.device_error() == 0


# 300 units leave a unit's tokens whole: 6400 of them into one sum
@pytest.mark.parametrize("B,H,N,d,dtype", [(300, 1, 6400, 64, "bf16"), (100, 3, 6401, 40, "bf16"), (300, 1, 4810, 64, "f32")])
def test_linear_orth_of_long_units_that_are_not_split(B, H, N, d, dtype):
    q, k, v = (randn(B, H, N, d, seed=s).div(d ** 0.5).to(DT[dtype]) for s in (1, 2, 3))
    w0 = randn(H, d, d, seed=4) / d ** 0.5
    out, w = ttt.linear_fullbatch_orth(q, k, v, w0, eta=0.2, with_w_star=True)
    units(q, k, v, w0, out, w, B, H)
