"""Sums of the layer norm's backward pass over many rows, so drawn that they are exact (GPU).

With dy of small whole numbers dbeta is a sum of whole numbers below 2^24, exact in fp32 in any order.  With rows
of +v and -v in equal numbers and eps = 0 the mean is 0 and the mean square v^2, both exact for a power of two v
and a row of 2^k features, and xh is +1 or -1 exactly (the reciprocal square root of a power of four is one of
a power of two): dgamma is such a sum too.  A row that is left out, taken twice or added to another column shows.
"""
import pytest
import torch

from linear_attention_split_b200 import ttt

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def draw(rows, C, dt, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    signs = torch.ones(rows, C, device=DEV)
    signs[:, C // 2:] = -1
    # every row its own order: a rotation by a place of its own
    at = torch.randint(C, (rows, 1), generator=g, device=DEV)
    signs = signs.gather(1, (torch.arange(C, device=DEV) + at) % C)
    v = 2.0 ** torch.randint(-3, 4, (rows, 1), generator=g, device=DEV)
    dy = torch.randint(-3, 4, (rows, C), generator=g, device=DEV).float()
    return (signs * v).to(dt), dy.to(dt), signs


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C", [(1, 64), (7, 8), (147, 256), (148 * 16, 256), (148 * 16 + 1, 256), (40000, 16), (12544, 512), (100001, 64),
                                    (6401, 2), (3000, 4096), (999, 8192), (300, 16384), (262144, 16)])
def test_weight_sums_miss_no_row(rows, C, dtype):
    x, dy, signs = draw(rows, C, DT[dtype], seed=rows + C)
    gamma = torch.ones(C, device=DEV)
    _, dgamma, dbeta = ttt.layernorm_bwd(dy, x, gamma, eps=0.0)
    assert torch.equal(dbeta, dy.double().sum(0).float())
    assert torch.equal(dgamma, (dy.double() * signs).sum(0).float())
    assert ttt.device_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [1, 3, 7, 33, 100, 257, 321, 385, 1000, 5000, 10000, 16383])
@pytest.mark.parametrize("rows", [1, 500, 5003])
def test_bias_sums_of_any_width(rows, C, dtype):
    # widths that no power of two describes: dbeta alone is exact
    g = torch.Generator(device=DEV).manual_seed(rows + C)
    dy = torch.randint(-3, 4, (rows, C), generator=g, device=DEV).to(DT[dtype])
    x = torch.randn(rows, C, generator=g, device=DEV).to(DT[dtype])
    dbeta = ttt.layernorm_bwd(dy, x, torch.ones(C, device=DEV))[2]
    assert torch.equal(dbeta, dy.double().sum(0).float())


def test_weight_sums_take_single_rows():
    # a gradient in one row only: its dgamma is that row's, wherever the row lies
    rows, C = 20011, 128
    x, _, signs = draw(rows, C, torch.bfloat16, seed=5)
    gamma = torch.ones(C, device=DEV)
    for row in (0, 1, 147, 148, 2367, 2368, 10007, rows - 2, rows - 1):
        dy = torch.zeros(rows, C, dtype=torch.bfloat16, device=DEV)
        dy[row] = torch.arange(C, device=DEV) - 60
        _, dgamma, dbeta = ttt.layernorm_bwd(dy, x, gamma, eps=0.0)
        assert torch.equal(dbeta, dy[row].float()) and torch.equal(dgamma, dy[row].float() * signs[row])


def test_weight_sums_past_32_bit_offsets():
    # 2^31 elements and a few rows
    rows, C = 524288 + 37, 4096
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GB of free device memory")
    x = torch.ones(rows, C, dtype=torch.bfloat16, device=DEV)
    x[:, 1::2] = -1
    dy = torch.ones(rows, C, dtype=torch.bfloat16, device=DEV)
    dy[524288 - 3:, ::7] = -2  # on both sides of the border
    _, dgamma, dbeta = ttt.layernorm_bwd(dy, x, torch.ones(C, device=DEV), eps=0.0)
    want = torch.full((C,), float(rows), dtype=torch.float64, device=DEV)
    want[::7] -= 3.0 * (rows - 524288 + 3)
    assert torch.equal(dbeta.double(), want)
    want[1::2] *= -1
    assert torch.equal(dgamma.double(), want)


WIDTHS = [*range(1, 140), *range(140, 600, 7), *range(600, 16384, 331), 255, 256, 257, 384, 385, 511, 512, 513, 1023, 1024, 1025, 2048,
          2052, 4096, 4097, 4100, 8191, 8192, 8193, 8196, 8200, 12000, 16368, 16376, 16380, 16383, 16384]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [3, 1200])
def test_every_width_has_its_kernels(rows, dtype):
    # dbeta of whole numbers is exact; y and dx of such rows against the definition
    g = torch.Generator(device=DEV).manual_seed(rows)
    for C in WIDTHS:
        x = torch.randn(rows, C, generator=g, device=DEV).to(DT[dtype])
        dy = torch.randint(-3, 4, (rows, C), generator=g, device=DEV).to(DT[dtype])
        gamma = torch.ones(C, device=DEV)
        y = ttt.layernorm(x, gamma, eps=1.0)
        dx, _, dbeta = ttt.layernorm_bwd(dy, x, gamma, eps=1.0)
        assert torch.equal(dbeta, dy.double().sum(0).float()), C
        c = x.double() - x.double().mean(1, keepdim=True)
        rstd = (c.square().mean(1, keepdim=True) + 1.0).rsqrt()
        xh, d = c * rstd, dy.double()
        want = rstd * (d - d.mean(1, keepdim=True) - xh * (d * xh).mean(1, keepdim=True))
        # a half step of the output for every value, and 64 roundings of fp32 of what a row's values reach (|xh| and
        # |dy| up to 8 here, rstd at most 1)
        h = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8
        assert ((y.double() - xh).abs() <= h * xh.abs() + 64 * 2.0 ** -24 * 8).all(), C
        assert ((dx.double() - want).abs() <= h * want.abs() + 64 * 2.0 ** -24 * 8 * 8).all(), C
    assert ttt.device_error() == 0
